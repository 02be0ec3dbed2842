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
template <int W>
struct FaShape {                                   // a CTA with W row tiles; 3 - W run on an SM
  static constexpr int STAGES = 2 * W;             // key stages
  static constexpr int THREADS = 128 + 128 * W;    // K producer, MMA, V producer, V cleaner | softmax A | softmax B
  static constexpr int SMEM = W * TILE + STAGES * 2 * TILE + 1024;
  static constexpr uint32_t COLS = 256 * W;        // tensor memory
};
constexpr uint32_t IDESC_S = tc::idesc_bf16(128, 128);
constexpr uint32_t IDESC_PV = tc::idesc_bf16(128, 64) | (1u << 16);   // B (V) is N-major
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
__device__ __forceinline__ int tile_entry(const AttnP& p, int t, int lane) {
  return p.geo.tpp ? t / p.geo.tpp : (t << p.geo.ppt_log) + lane;
}
__device__ __forceinline__ int tile_page(const AttnP& p, const int32_t* table, int t, int lane) {
  const int e = tile_entry(p, t, lane);
  return (p.geo.tpp || lane < (1 << p.geo.ppt_log)) && e < p.c.table_stride ? __ldg(table + e) : -1;
}
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
    f.tok = 0;
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
  uint64_t q_full[W], full[FaShape<W>::STAGES], empty[FaShape<W>::STAGES], raw[FaShape<W>::STAGES], s_full[W], s_free[W],
      p_full[W], pv_done[W];
};

template <int W>
__global__ void __launch_bounds__(FaShape<W>::THREADS, 3 - W)
fa_kernel(const AttnP p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mv) {
  constexpr int NST = FaShape<W>::STAGES, THREADS = FaShape<W>::THREADS;
  constexpr uint32_t TM_S = 0, TM_P = 128 * W, TM_O = 192 * W;   // + 128 w, + 64 w, + 64 w
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) Bars<W> B;
  __shared__ Meta meta[NST];
  __shared__ Odd odd;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  if (p.next_item && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *p.next_item = 0ull;
  const int groups = (p.row_tiles + W - 1) / W;
  const int pair = groups - 1 - blockIdx.x / p.nsplit, split = blockIdx.x % p.nsplit;   // the longest rows first
  const int h = blockIdx.y, i = longest_first(p, blockIdx.z);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Req r = request(p, i);
  const int R = r.c * p.G, RB = FA_ROWS / p.G, TR = RB * p.G;
  const int rho0 = pair * W * TR;
  if (rho0 >= R) return;
  // key tiles of each row tile within this split
  int n[W], lo;
  {
    const int ps = p.c.page_size;
    lo = split * p.tps;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int first = rho0 + w * TR, last = min(R, first + TR) - 1;
      const int nt = last >= first ? tile_count(p.geo, ps, FA_KEYS, row_limit(p, r, last / p.G)) : 0;
      n[w] = max(0, min(nt, lo + p.tps) - lo);
    }
  }
  const int nmax = max(n[0], n[W - 1]);
  volatile int* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int b = 0; b < NST; ++b) {
      tc::mbar_init(&B.full[b], 2);
      tc::mbar_init(&B.empty[b], 1);
      tc::mbar_init(&B.raw[b], 1);
    }
    odd.any = 0;
    for (int w = 0; w < W; ++w) {
      tc::mbar_init(&B.q_full[w], 1); tc::mbar_init(&B.s_full[w], 1); tc::mbar_init(&B.s_free[w], 4);
      tc::mbar_init(&B.p_full[w], 4); tc::mbar_init(&B.pv_done[w], 1);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tc::tmem_alloc(&s_tmem, FaShape<W>::COLS);
  uint8_t* sQ = sm;
  auto sK = [&](int b) { return sm + W * TILE + b * 2 * TILE; };
  auto sV = [&](int b) { return sm + (W + 1) * TILE + b * 2 * TILE; };
  if (p.geo.tpp && p.geo.box < FA_KEYS)            // value rows that no copy writes
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
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0 || warp == 2) {
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
  } else if (warp == 3) {
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
      const int s = j % NST;
      if ((w == 0 || j >= n[0]) && !wait(&B.full[s], (uint32_t)((j / NST) & 1), abort)) return false;
      if (j > 0 && !wait(&B.s_free[w], (uint32_t)((j - 1) & 1), abort)) return false;
      tc::tc_fence_after();
      if (lead) {
        const uint64_t qd = qd0 + (uint64_t)(w * (TILE >> 4)), kd = kd0 + (uint64_t)(s * (2 * TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < WS_DH / 16; ++kk)
          tc::umma_bf16(tmem + TM_S + 128u * w, qd + (uint64_t)(kk * 2), kd + (uint64_t)(kk * 2), IDESC_S, kk ? 1u : 0u);
        tc::umma_commit(&B.s_full[w]);
      }
      __syncwarp();
      return true;
    };
    auto pv = [&](int w, int j) -> bool {
      const int s = j % NST;
      if (!wait(&B.p_full[w], (uint32_t)(j & 1), abort)) return false;
      tc::tc_fence_after();
      if (lead) {
        const uint64_t vd = vd0 + (uint64_t)(s * (2 * TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < FA_KEYS / 16; ++kk)
          umma_ts(tmem + TM_O + 64u * w, tmem + TM_P + 64u * w + 8u * kk, vd + (uint64_t)(kk * 128), IDESC_PV,
                  (j | kk) ? 1u : 0u);
        tc::umma_commit(&B.pv_done[w]);
        if (w == W - 1 || j >= n[W - 1]) tc::umma_commit(&B.empty[s]);     // the stage's last reader
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
  } else {
    // ---- softmax: thread = row
    if (W == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");     // 168 a thread at launch
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");            // 128
    const int w = (warp >> 2) - 1, quarter = warp & 3, x = quarter * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tS = tl + TM_S + 128u * w, tP = tl + TM_P + 64u * w, tO = tl + TM_O + 64u * w;
    const int first = rho0 + w * TR, rho = first + x;
    const bool on = x < TR && rho < R;
    const int t = on ? rho / p.G : 0;
    const int lim = on ? row_limit(p, r, t) : 0, lim_all = first < R ? row_limit(p, r, first / p.G) : 0;
    const float sl = p.sl;
    const float2 sl2 = make_float2(sl, sl);
    float m = -INFINITY, msl = 0.f, l = 0.f;
    bool ok = true;
    const int nw = n[w];
    for (int j = 0; j < nw; ++j) {
      if (!wait_warp(&B.s_full[w], (uint32_t)(j & 1), abort)) { ok = false; break; }
      tc::tc_fence_after();
      float sv[FA_KEYS];
#pragma unroll
      for (int q = 0; q < 8; ++q) tm_ld16(tS + 16 * q, sv + 16 * q);
      const Meta& mt = meta[j % NST];
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
      float2 sum2[2];
      auto weigh = [&]() {
        const float2 nm2 = make_float2(-msl, -msl);
        sum2[0] = sum2[1] = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = __ffma2_rn(make_float2(sv[32 * q + 2 * e], sv[32 * q + 2 * e + 1]), sl2, nm2);
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
      if (j > 0) tile = weigh();
      if (j == 0 || __any_sync(0xffffffffu, on && (m == -INFINITY || !(tile < MOST)))) {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < FA_KEYS; e += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], sv[e + 2 * q], sv[e + 2 * q + 1]);
        const float mn = fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
        const float f = m > -INFINITY ? ex2((m - mn) * sl) : (mn > -INFINITY ? 0.f : 1.f);
        m = mn;
        msl = mn > -INFINITY ? mn * sl : 0.f;
        l *= f;
        if (j > 0) {
          st_wait();                               // the first weights are stored before the second ones are
          tc::tc_fence_after();
#pragma unroll
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
    const bool any_odd = nw > 0 && *(volatile int*)&odd.any != 0;
    if (p.nsplit > 1) {
      const size_t at = on ? (((size_t)i * p.c.n_kv_heads + h) * ((size_t)p.a.max_q * p.G) + rho) * p.nsplit + split : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float o[16];
        if (nw > 0) { tm_ld16(tO + 16 * q, o); ld_wait(); }
        if (any_odd)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = with_odd(odd, o[e], lim, 16 * q + e);
        if (on)
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(p.part_o + at * WS_DH + 16 * q + e) =
                nw > 0 ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (on) p.part_ml[at] = make_float2(m == -INFINITY ? m : msl, ok ? l : NAN);
    } else {
      const float inv = !ok ? NAN : l == 0.f ? 0.f : 1.f / l;
      const int u_ = h * p.G + (on ? rho - t * p.G : 0);
      bf16* out = (bf16*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u_ * WS_DH;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float o[16];
        if (nw > 0) { tm_ld16(tO + 16 * q, o); ld_wait(); }
        if (any_odd)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = with_odd(odd, o[e], lim, 16 * q + e);
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
  if (warp == 1) tc::tmem_dealloc(tmem, FaShape<W>::COLS);
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

template <int W>
cudaError_t run_fa(const AttnP& p, const TcMap& mq, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(fa_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, FaShape<W>::SMEM);
  if (e != cudaSuccess) return e;
  fa_kernel<W><<<dim3((p.row_tiles + W - 1) / W * p.nsplit, p.c.n_kv_heads, p.a.n_req), FaShape<W>::THREADS, FaShape<W>::SMEM, s>>>(
      p, reinterpret_cast<const CUtensorMap&>(mq), reinterpret_cast<const CUtensorMap&>(mk),
      reinterpret_cast<const CUtensorMap&>(mv));
  ws_count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fa(const AttnP& p, cudaStream_t s) {
  TcMap mq, mk, mv;
  if (!tc_encode_heads(&mq, p.a.q, p.a.q_stride, (uint64_t)p.a.total_q, (uint32_t)p.a.n_heads, (uint32_t)p.G,
                       (uint32_t)(FA_ROWS / p.G)) ||
      !tc_encode_paged(&mk, p.c.k, p.c, (uint32_t)p.geo.box) || !tc_encode_paged(&mv, p.c.v, p.c, (uint32_t)p.geo.box))
    return cudaErrorInvalidValue;
  return p.row_tiles == 1 ? run_fa<1>(p, mq, mk, mv, s) : run_fa<2>(p, mq, mk, mv, s);
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

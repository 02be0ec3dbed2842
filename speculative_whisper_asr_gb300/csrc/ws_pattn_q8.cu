// Attention over a cache in 8 bits (e4m3 values, a power of two per block of
// tokens and head), few rows: the cache is streamed once.
//
// One CTA takes a tile of up to 8 * NT rows and a range of key tiles; its four
// warps take every fourth tile of 32 keys through private rings of TMA slots,
// and the products are taken transposed, as for bf16 (ws_pattn.cu):
//   S^T = K Q^T    (16 keys x 8 rows per mma m16n8k16),
//   O^T = V^T P^T  (16 dims x 8 rows).
// Half the bytes per element leave half the time per element, so the codes go
// from shared memory through one conversion (two e4m3 to two fp16, exact)
// straight into matrix operands.  For that the dims and keys are dealt out so
// that a lane's operand is what lies together:
//   - S: a dot product does not care which dim stands at which k, so lane c
//     of a quad takes dims 16 c .. 16 c + 15 of its key: one 16-byte read.
//   - O: lane g holds dims 8 g .. 8 g + 7 of its keys (8-byte reads); a byte
//     permutation puts the same dim of two keys side by side.  Place p of a
//     tile's S holds the tile's key KEY(p), a reordering by which the 16 lanes
//     of a read fall into different banks of the 64-byte swizzle.
// Scales never touch an element: a key's multiplies its scores (fp32), a
// value's its weight.  Weights enter the product as fp16, 2^-11 of each at
// most, an eighth of the bf16 output's own step, relative to 2^E, the largest
// value scale that the row has seen so far, so that they stay within fp16
// whatever the scales are.  They are at most 2^8 and stored 2^7 times larger, so
// that fp16's last step is 2^-31 of a row's largest weight times the largest
// value scale.  Queries, 8 bits each, are exact in fp16 once a row's largest is
// brought to 1 .. 2 by a power of two, which joins the row's scale; elements
// below 2^-17 of the largest round to 2^-25 of it, the step of the fp32 sums.
//
// 16 requests x 1 row, 32 heads on 8, up to 65,536 positions (680 MB): 132 us,
// 5.1 TB/s; the copies alone take 117.  96 x 9 rows, 20 heads, 375-1500
// positions (234 MB): 71 us, 3.3 TB/s; the copies alone take 54, because a
// CTA has a dozen microseconds of work between its rings' first fill and the
// join of its warps.  Two CTAs per SM with 6 slots per warp 90 and 162 us, 8
// warps 81 in the second, four CTAs per SM spill.  Above 16 rows the products
// bound it: 85 / 128 / 174 us at 17 / 32 / 48 rows.
#include <type_traits>

#include "ws_pattn.cuh"

namespace {

constexpr int TK = Q8_TK;
constexpr int W = 4;                       // warps
constexpr int NS = 4;                      // ring slots per warp
constexpr int TB = TK * WS_DH;             // bytes of a K or V tile
constexpr int OP = WS_DH + 4;              // row pitch of the CTA's merge area, which reuses the rings
constexpr float HOLD = 8.0f;               // log2 of the largest weight before a row's reference moves
constexpr float RAISE = 128.0f;            // weights are stored this much larger
constexpr int q8_smem(int nt) {
  const int ring = W * NS * 2 * TB, merge = W * 8 * nt * (OP + 2) * 4;
  return (ring > merge ? ring : merge) + 1024;
}

struct Slot {                              // of a ring: keys that count, the first position, bytes of the keys' scales
  uint32_t valid;
  int base;
  uint8_t ks[TK], vs[TK];                  // UNI: of all keys, in place 0
};
// Key of a 32-key tile that stands at place p of the products: bits 0 and 1 of
// it change places, so that the keys of a quad's lanes (bits 1 and 2 of p)
// differ in bits 0 and 2, which choose the half line and the swizzle's line half.
__device__ __forceinline__ int KEY(int p) { return (p & ~3) | (p & 1) << 1 | (p >> 1 & 1); }

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// 2^e for e <= 0 (0 below fp32's normal numbers).
__device__ __forceinline__ float down(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(e + 127) << 23); }

// NaN codes among a value tile's rows (lane = row), noted and cleared.
__device__ __noinline__ void note_nan(Odd& odd, uint8_t* row, int r, int pos, int lane) {
  if (!odd.any)
    for (int x = lane; x < 3 * WS_DH; x += 32) odd.first[0][x] = 0x7FFFFFFF;
  __syncwarp();
  for (int b = 0; b < WS_DH; ++b)
    if ((row[b] & 0x7Fu) == 0x7Fu) {
      atomicMin(&odd.first[2][((b >> 4) ^ ((r >> 1) & 3)) * 16 + (b & 15)], pos);
      row[b] = 0;
    }
  __syncwarp();
  if (lane == 0) odd.any = 1;
}
// True if there were any.
__device__ __forceinline__ bool take_out_nan(Odd& odd, uint8_t* tile, int base, int lane) {
  uint32_t found = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 v = reinterpret_cast<const uint4*>(tile + lane * WS_DH)[q];
    found |= ((v.x & 0x7F7F7F7Fu) + 0x01010101u) | ((v.y & 0x7F7F7F7Fu) + 0x01010101u) |
             ((v.z & 0x7F7F7F7Fu) + 0x01010101u) | ((v.w & 0x7F7F7F7Fu) + 0x01010101u);
  }
  if (!__any_sync(0xffffffffu, (found & 0x80808080u) != 0u)) return false;
  note_nan(odd, tile + lane * WS_DH, lane, base + lane, lane);
  return true;
}

// MIX: causal chunks of more than one row, where NaN values are kept from the
// rows that do not see them.  UNI: scales hold for whole tiles (blocks of 32;
// 71 us for the second call above, 75 in blocks of 16 or 8).
template <int NT, bool MIX, bool UNI>
__global__ void __launch_bounds__(W * 32, 3)
q8_kernel(const AttnP p, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  constexpr int MT = TK / 16;              // key steps of 16
  constexpr uint32_t ALL = 0xffffffffu;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t full[W][NS];
  __shared__ __align__(16) Slot slots[W][NS];
  __shared__ Odd odd[MIX ? W : 1];         // each warp's own
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rt = blockIdx.x / p.nsplit, split = blockIdx.x - rt * p.nsplit, h = blockIdx.y, i = blockIdx.z;
  pdl_trigger();
  // the first tiles' pages are asked for together with the lengths: the
  // entries exist whatever the lengths turn out to be
  const int slot0 = p.a.req_ids ? p.a.req_ids[i] : i;
  const int32_t* table = p.c.page_table + (size_t)min(max(slot0, 0), p.c.n_slots - 1) * p.c.table_stride;
  TileWalk w;
  auto page_of = [&]() -> int {            // table entry of this lane's key in the walk's tile, -1: none
    int e = w.entry(p.geo, lane);
    if (!UNI && p.geo.pieces > 1) e /= p.geo.pieces;
    return e < p.c.table_stride ? __ldg(table + e) : -1;
  };
  w.start(p.geo, split * p.tps + warp, W);
  int page0[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) { page0[s] = page_of(); w.next(p.geo); }
  const Req r = request(p, i);
  const int R = r.c * p.G, r0 = rt * 8 * NT;
  if (r0 >= R) return;
  if (lane == 0)
    for (int s = 0; s < NS; ++s) tc::mbar_init(&full[warp][s], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  // positions that some row of this tile sees, and those that all see
  const int last = min(R, r0 + 8 * NT) - 1;
  const int Lmax = row_limit(p, r, last / p.G), Lmin = row_limit(p, r, r0 / p.G);
  const int nt_all = tile_count(p.geo, p.c.page_size, TK, Lmax);
  const int tb = min(nt_all, split * p.tps), te = min(nt_all, tb + p.tps);
  const int n_my = max(0, (te - tb - warp + W - 1) / W);
  uint8_t* ring = sm + warp * (NS * 2 * TB);
  uint32_t k_byte, v_byte;                 // scales of this lane's key in the tile asked for last
  const uint8_t* k_scales = p.c.k_scale + (size_t)h * (size_t)p.c.scale_head_stride;
  const uint8_t* v_scales = p.c.v_scale + (size_t)h * (size_t)p.c.scale_head_stride;
  auto issue = [&](int slot, int page) {
    const int base = w.base(p.geo, p.c.page_size, TK);
    const bool ok = page >= 0 && page < p.c.n_pages && lane < w.room(p.geo, p.c.page_size, TK) && base + lane < Lmax;
    const uint32_t valid = __ballot_sync(ALL, ok);
    const bool go = ok && (p.geo.tpp ? (valid & ((1u << lane) - 1u)) == 0u : (lane & (p.geo.box - 1)) == 0);
    const unsigned boxes = __ballot_sync(ALL, go);
    if (lane == 0) {
      slots[warp][slot].valid = valid;
      slots[warp][slot].base = base;
      tc::mbar_expect_tx(&full[warp][slot], (uint32_t)__popc(boxes) * 2u * (uint32_t)p.geo.box * (uint32_t)WS_DH);
    }
    __syncwarp();
    // several pages: first token of this lane's copy
    const int tok0 = !UNI && p.geo.pieces > 1 ? w.entry(p.geo, lane) % p.geo.pieces * p.geo.box : 0;
    if (go) {
      uint8_t* dst = ring + slot * (2 * TB) + (p.geo.tpp ? 0 : lane * WS_DH);
      const int tok = p.geo.tpp ? w.sub * TK : tok0;
      tma_load_4d(dst, &mk, &full[warp][slot], 0, tok, h, page);
      tma_load_4d(dst + TB, &mv, &full[warp][slot], 0, tok, h, page);
    }
    k_byte = v_byte = 0;
    if (ok) {
      const uint32_t tok = (uint32_t)(p.geo.tpp ? w.sub * TK + (UNI ? 0 : lane) : tok0 + (lane & (p.geo.box - 1)));
      uint32_t b = p.block_mul ? __umulhi(tok, p.block_mul) : tok;        // tok / scale_block, or one more
      b -= b * (uint32_t)p.c.scale_block > tok;
      const uint64_t at = (uint64_t)(uint32_t)page * (uint32_t)p.c.scale_page_stride + b;
      k_byte = __ldg(k_scales + at);
      v_byte = __ldg(v_scales + at);
    }
  };
  // A slot's scales are stored a tile after they were asked for.
  auto keep_scales = [&](int slot) {
    if (UNI) {                             // of any key that counts: a tile of one scale is a tile of one page
      const uint32_t kb = __reduce_max_sync(ALL, k_byte), vb = __reduce_max_sync(ALL, v_byte);
      if (lane == 0) {
        slots[warp][slot].ks[0] = (uint8_t)kb;
        slots[warp][slot].vs[0] = (uint8_t)vb;
      }
    } else {
      slots[warp][slot].ks[lane] = (uint8_t)k_byte;
      slots[warp][slot].vs[lane] = (uint8_t)v_byte;
    }
  };
  w.start(p.geo, split * p.tps + warp, W);
  uint32_t first_k[NS], first_v[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s)
    if (s < n_my) {
      issue(s, page0[s]);
      w.next(p.geo);
      first_k[s] = k_byte;
      first_v[s] = v_byte;
    }
#pragma unroll
  for (int s = 0; s < NS; ++s)             // behind the last copy: they wait for the scales
    if (s < n_my) {
      k_byte = first_k[s];
      v_byte = first_v[s];
      keep_scales(s);
    }
  int page_next = page_of();               // of the tile asked for next: looked up a tile ahead

  // ---- queries: rows r0 + 8 nt + g, dims 16 c .. 16 c + 15 of this lane
  uint32_t qf[4][NT][2];
  float sl[NT][2];                         // of this lane's rows 8 nt + 2 c + e: score scale in log2 units
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rho = r0 + 8 * nt + g;
    const bool on = rho < R;
    const int t = on ? rho / p.G : 0;
    const bf16* q = (const bf16*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride + (size_t)(h * p.G + (on ? rho - t * p.G : 0)) * WS_DH + 16 * c;
    uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (on) {
      v[0] = __ldg(reinterpret_cast<const uint4*>(q));
      v[1] = __ldg(reinterpret_cast<const uint4*>(q) + 1);
    }
    const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    float x[16], most = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = (u[k] & p.q_and) ^ p.q_xor;
      x[2 * k] = __uint_as_float(b << 16);
      x[2 * k + 1] = __uint_as_float(b & 0xFFFF0000u);
      most = fmaxf(most, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1])));
    }
    most = fmaxf(most, __shfl_xor_sync(ALL, most, 1));
    most = fmaxf(most, __shfl_xor_sync(ALL, most, 2));
    // 2^-e and 2^e, e the exponent of the largest; rows of zeros, of numbers below fp32's normal ones, or with
    // infinities stay as they are
    const int e = most >= 1.17549435e-38f && most < INFINITY ? min((int)(__float_as_uint(most) >> 23) - 127, 126) : 0;
    const float f = __uint_as_float((uint32_t)(127 - e) << 23), back = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int k = 0; k < 2; ++k) qf[s][nt][k] = pack_f16(x[4 * s + 2 * k] * f, x[4 * s + 2 * k + 1] * f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sl[nt][k] = score_factor(p.sl * __shfl_sync(ALL, back, 4 * (2 * c + k)));
    }
  }
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) lim[nt][e] = row_limit(p, r, min(r0 + 8 * nt + 2 * c + e, R - 1) / p.G);
  float o[4][NT][4], m[NT][2], l[NT][2];   // m: the rows' references, in log2 units
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) { m[nt][e] = -INFINITY; l[nt][e] = 0.f; }
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][nt][e] = 0.f;
  }
  int E[MIX ? NT : 1][MIX ? 2 : 1] = {};   // byte of the largest value scale that the rows have seen so far
  const bool mixed = MIX && Lmin < Lmax;   // some row does not see all of the tile's positions
  if (MIX && lane == 0) odd[warp].any = 0;
  const int key_g = KEY(g), key_c = KEY(2 * c);            // of places g and 2 c
  bool dead = false;
  auto tile = [&](int it, auto last_tiles) -> bool {
    const int slot = it % NS;
    if (!tc::mbar_wait(&full[warp][slot], (uint32_t)((it / NS) & 1))) { dead = true; return false; }
    __syncwarp();
    const Slot& sl_ = slots[warp][slot];
    const uint32_t valid = sl_.valid;
    const int base = sl_.base;
    uint8_t* Kt = ring + slot * (2 * TB);
    uint8_t* Vt = Kt + TB;
    if (valid != ALL) {
      // rows that do not count may hold anything: 0 * NaN would reach the sums
      if (!((valid >> lane) & 1u)) {
#pragma unroll
        for (int q = 0; q < 4; ++q) reinterpret_cast<uint4*>(Vt + lane * WS_DH)[q] = make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the slot's next copy
      __syncwarp();
    }
    if (decltype(last_tiles)::value && take_out_nan(odd[warp], Vt, base, lane)) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    }
    // ---- the tile into registers, so that its slot takes the next copy at once:
    // what is under way bounds the rate (slots held until the end: 141 us for 117)
    const uint32_t kb = tc::smem_u32(Kt), vb = tc::smem_u32(Vt);
    uint4 kw[MT][2];                       // key 16 mt + 8 e2 + key_g, dims 16 c ..
    uint2 vw[MT][2][2];                    // keys 16 mt + 8 e2 + key_c, + 2 (places 2 c, 2 c + 1), dims 8 g ..
    int vs[MT][2];                         // scales of the former keys' values, and of them
    float ksc[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const int key = 16 * mt + 8 * e2 + key_g, k0 = 16 * mt + 8 * e2 + key_c;
        kw[mt][e2] = lds128(kb + key * WS_DH + ((c ^ ((key >> 1) & 3)) << 4));
#pragma unroll
        for (int e = 0; e < 2; ++e)
          vw[mt][e2][e] = lds64(vb + (k0 + 2 * e) * WS_DH + (((g >> 1) ^ (((k0 + 2 * e) >> 1) & 3)) << 4) + ((g & 1) << 3));
        if (!UNI || (mt == 0 && e2 == 0)) {
          vs[mt][e2] = sl_.vs[UNI ? 0 : key];
          ksc[mt][e2] = scale_of(sl_.ks[UNI ? 0 : key]);
        }
      }
    __syncwarp();                          // every lane has read the slot
    // the scales asked for at the end of the last tile, of the slot that it freed
    if (it > 0 && it - 1 + NS < n_my) keep_scales((it - 1) % NS);
    if (it + NS < n_my) {
      issue(slot, page_next);
      w.next(p.geo);
      page_next = page_of();
    }
    // ---- S^T: place 16 mt + 8 e2 + g of the products is key 16 mt + 8 e2 + key_g
    float sc[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t a[4][4];
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        widen(kw[mt][e2].x, a[0][e2], a[0][2 + e2]);
        widen(kw[mt][e2].y, a[1][e2], a[1][2 + e2]);
        widen(kw[mt][e2].z, a[2][e2], a[2][2 + e2]);
        widen(kw[mt][e2].w, a[3][e2], a[3][2 + e2]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_f16(sc[mt][nt], a[s], qf[s][nt][0], qf[s][nt][1]);
      }
      if (!UNI)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) { sc[mt][nt][2 * e2] *= ksc[mt][e2]; sc[mt][nt][2 * e2 + 1] *= ksc[mt][e2]; }
    }
    if (valid != ALL || base + TK > Lmin) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int j = 16 * mt + 8 * e2 + key_g;
          const bool ok = (valid >> j) & 1u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!ok || base + j >= lim[nt][e]) sc[mt][nt][2 * e2 + e] = -INFINITY;
        }
    }
    // ---- a larger value scale than before?  The same for all rows as long as
    // they see the same; then each row's own, of the keys that it sees: a scale
    // that it does not see would take its weights' last bits, or all of them.
    constexpr bool OWN = MIX && decltype(last_tiles)::value;
    const int most = UNI ? vs[0][0] : max(max(vs[0][0], vs[0][1]), max(vs[1][0], vs[1][1]));
    int least = E[0][0];                   // of this lane's rows
    if (OWN)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) least = min(least, E[MIX ? nt : 0][MIX ? e : 0]);
    const bool larger = __any_sync(ALL, most > least);
    if (OWN && larger) {
      int now[NT][2];
      bool more = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          now[nt][e] = E[MIX ? nt : 0][MIX ? e : 0];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int j = 16 * mt + 8 * e2 + key_g, s = UNI ? vs[0][0] : vs[mt][e2];
              if (((valid >> j) & 1u) && base + j < lim[nt][e] && s > now[nt][e]) { now[nt][e] = s; more = true; }
            }
        }
      if (__any_sync(ALL, more)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int t = now[nt][e];
            t = max(t, __shfl_xor_sync(ALL, t, 4));
            t = max(t, __shfl_xor_sync(ALL, t, 8));
            t = max(t, __shfl_xor_sync(ALL, t, 16));
            int& was = E[MIX ? nt : 0][MIX ? e : 0];
            const float f = down(was - t);
            was = t;
#pragma unroll
            for (int d = 0; d < 4; ++d) { o[d][nt][e] *= f; o[d][nt][2 + e] *= f; }
          }
      }
    } else if (larger) {
      const int now = UNI ? most : __reduce_max_sync(ALL, max(most, least));
      const float f = down(least - now);
#pragma unroll
      for (auto& row : E)
#pragma unroll
        for (int& x : row) x = now;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][nt][e] *= f;
    }
    // ---- does a score pass its row's reference by more than 2^8?
    bool grow = false;
    float slk[NT][2], top[NT][2];          // UNI: with the keys' scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        slk[nt][e] = UNI ? score_factor(sl[nt][e] * ksc[0][0]) : sl[nt][e];
        top[nt][e] = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e])) * slk[nt][e];
        grow |= top[nt][e] > m[nt][e] + HOLD;
      }
    if (__any_sync(ALL, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t4 = top[nt][e];
          t4 = fmaxf(t4, __shfl_xor_sync(ALL, t4, 4));
          t4 = fmaxf(t4, __shfl_xor_sync(ALL, t4, 8));
          t4 = fmaxf(t4, __shfl_xor_sync(ALL, t4, 16));
          const float mn = t4 > m[nt][e] + HOLD ? t4 : m[nt][e];
          const float f = m[nt][e] > -INFINITY ? ex2(m[nt][e] - mn) : 0.f;
          m[nt][e] = mn;
          l[nt][e] *= f;
#pragma unroll
          for (int d = 0; d < 4; ++d) { o[d][nt][e] *= f; o[d][nt][2 + e] *= f; }
        }
    }
    float ref[NT][2];                      // 0 where a row has none yet
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) ref[nt][e] = m[nt][e] > -INFINITY ? m[nt][e] : 0.f;
    uint32_t pf[MT][NT][2];
    // a weight's factor; keys that a row does not see have weight 0, whatever their scale
    auto factor = [&](int s, int nt, int e) { return down(OWN ? min(s - E[MIX ? nt : 0][MIX ? e : 0], 0) : s - E[0][0]) * RAISE; };
    float fu[NT][2] = {};                  // UNI: of all keys
    if (UNI)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) fu[nt][e] = factor(vs[0][0], nt, e);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float p0 = ex2(fmaf(sc[mt][nt][2 * e2], slk[nt][0], -ref[nt][0]));
          const float p1 = ex2(fmaf(sc[mt][nt][2 * e2 + 1], slk[nt][1], -ref[nt][1]));
          l[nt][0] += p0;
          l[nt][1] += p1;
          pf[mt][nt][e2] = movm(pack_f16(p0 * (UNI ? fu[nt][0] : factor(vs[mt][e2], nt, 0)), p1 * (UNI ? fu[nt][1] : factor(vs[mt][e2], nt, 1))));
        }
      }
    // ---- O^T: dims 8 g + 2 d (rows 0 .. 7 of step d) and 8 g + 2 d + 1 (rows 8 .. 15)
#pragma unroll
    for (int ks = 0; ks < MT; ++ks) {
      uint32_t a[4][4];
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        const uint2 v0 = vw[ks][e2][0], v1 = vw[ks][e2][1];
        widen(__byte_perm(v0.x, v1.x, 0x5140), a[0][2 * e2], a[0][2 * e2 + 1]);
        widen(__byte_perm(v0.x, v1.x, 0x7362), a[1][2 * e2], a[1][2 * e2 + 1]);
        widen(__byte_perm(v0.y, v1.y, 0x5140), a[2][2 * e2], a[2][2 * e2 + 1]);
        widen(__byte_perm(v0.y, v1.y, 0x7362), a[3][2 * e2], a[3][2 * e2 + 1]);
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[d][nt], a[d], pf[ks][nt][0], pf[ks][nt][1]);
    }
    return true;
  };
  int it = 0;
  if (MIX) {
    // this warp's tiles that end at or before Lmin
    const int whole = tile_whole(p.geo, p.c.page_size, TK, Lmin);
    const int n_whole = mixed ? min(n_my, max(0, (whole - tb - warp + W - 1) / W)) : n_my;
    while (it < n_whole && tile(it, std::false_type())) ++it;
    while (!dead && it < n_my && tile(it, std::true_type())) ++it;
  } else {
    while (it < n_my && tile(it, std::false_type())) ++it;
  }
  // ---- the four warps' partials meet in shared memory
  __syncthreads();
  float* so = reinterpret_cast<float*>(sm);                // [warp][8 NT][OP]
  float* sml = so + W * 8 * NT * OP;                       // [warp][8 NT][2]: reference in log2 units, sum
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[nt][e];
      s += __shfl_xor_sync(ALL, s, 4);
      s += __shfl_xor_sync(ALL, s, 8);
      s += __shfl_xor_sync(ALL, s, 16);
      const int row = 8 * nt + 2 * c + e;
      const float size = scale_of((uint32_t)E[MIX ? nt : 0][MIX ? e : 0]) * (1.0f / RAISE);
      float* dst = so + (warp * 8 * NT + row) * OP;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        *reinterpret_cast<float2*>(dst + 8 * g + 2 * d) = make_float2(o[d][nt][e] * size, o[d][nt][2 + e] * size);
      if (g == 0) {
        sml[(warp * 8 * NT + row) * 2] = dead ? NAN : m[nt][e];
        sml[(warp * 8 * NT + row) * 2 + 1] = dead ? NAN : s;
      }
    }
  __syncthreads();
  if (MIX && (odd[0].any | odd[MIX ? 1 : 0].any | odd[MIX ? 2 : 0].any | odd[MIX ? 3 : 0].any)) {
    for (int x = threadIdx.x; x < W * 8 * NT * WS_DH; x += W * 32) {
      const int k = x / (8 * NT * WS_DH), row = x / WS_DH % (8 * NT), d = x % WS_DH;
      if (r0 + row >= R || !odd[k].any) continue;
      if (row_limit(p, r, (r0 + row) / p.G) > odd[k].first[2][d]) so[(k * 8 * NT + row) * OP + d] = NAN;
    }
    __syncthreads();
  }
  for (int x = threadIdx.x; x < 8 * NT * 16; x += W * 32) {
    const int row = x >> 4, d4 = x & 15, rho = r0 + row;
    if (rho >= R) continue;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) M = fmaxf(M, sml[(k * 8 * NT + row) * 2]);
    float sum = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float mk_ = sml[(k * 8 * NT + row) * 2];
      const float f = mk_ == -INFINITY ? 0.f : ex2(mk_ - M);
      const float4 v = *reinterpret_cast<const float4*>(so + (k * 8 * NT + row) * OP + 4 * d4);
      sum = fmaf(f, sml[(k * 8 * NT + row) * 2 + 1], sum);
      a0 = fmaf(f, v.x, a0); a1 = fmaf(f, v.y, a1); a2 = fmaf(f, v.z, a2); a3 = fmaf(f, v.w, a3);
    }
    if (p.nsplit > 1) {
      const size_t at = (((size_t)i * p.c.n_kv_heads + h) * ((size_t)p.a.max_q * p.G) + rho) * p.nsplit + split;
      *reinterpret_cast<float4*>(p.part_o + at * WS_DH + 4 * d4) = make_float4(a0, a1, a2, a3);
      if (d4 == 0) p.part_ml[at] = make_float2(M, sum);
      continue;
    }
    const int t = rho / p.G, u = h * p.G + rho - t * p.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(a0 * inv, a1 * inv), b1 = __floats2bfloat162_rn(a2 * inv, a3 * inv);
    bf16* out = (bf16*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u * WS_DH + 4 * d4;
    *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    if (p.lse && d4 == 0) p.lse[(size_t)(r.row0 + t) * p.a.n_heads + u] = sum == 0.f ? -INFINITY : (M + lg2(sum)) * LN2;
  }
  // a wait that ran out leaves copies in flight: see them land before the memory is given back
  if (dead)
    for (int s = 0; s < NS; ++s) { tc::mbar_wait(&full[warp][s], 0); tc::mbar_wait(&full[warp][s], 1); }
}

template <int NT, bool MIX, bool UNI>
cudaError_t run(const AttnP& p, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(q8_kernel<NT, MIX, UNI>, cudaFuncAttributeMaxDynamicSharedMemorySize, q8_smem(NT));
  if (e != cudaSuccess) return e;
  q8_kernel<NT, MIX, UNI><<<dim3(p.row_tiles * p.nsplit, p.c.n_kv_heads, p.a.n_req), W * 32, q8_smem(NT), s>>>(
      p, reinterpret_cast<const CUtensorMap&>(mk), reinterpret_cast<const CUtensorMap&>(mv));
  ws_count_launches(1);
  return cudaGetLastError();
}
template <bool MIX, bool UNI>
cudaError_t run(const AttnP& p, int nt, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  return nt == 1 ? run<1, MIX, UNI>(p, mk, mv, s) : run<2, MIX, UNI>(p, mk, mv, s);
}

}  // namespace

cudaError_t launch_q8(const AttnP& p, int nt, cudaStream_t s) {
  TcMap mk, mv;
  if (!tc_encode_paged(&mk, p.c.k, p.c, (uint32_t)p.geo.box) || !tc_encode_paged(&mv, p.c.v, p.c, (uint32_t)p.geo.box))
    return cudaErrorInvalidValue;
  const bool mix = p.a.causal && p.a.max_q > 1, uni = p.c.scale_block % TK == 0;
  if (mix) return uni ? run<true, true>(p, nt, mk, mv, s) : run<true, false>(p, nt, mk, mv, s);
  return uni ? run<false, true>(p, nt, mk, mv, s) : run<false, false>(p, nt, mk, mv, s);
}

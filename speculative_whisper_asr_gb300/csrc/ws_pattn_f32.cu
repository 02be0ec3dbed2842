// ws_paged_attention for the fp32 model: everything in fp32 on the FMA pipes
// (the tensor cores have no fp32 product).
//
// f32_kernel.  One CTA of 256 threads per (request, KV head, row tile of
// 16 * RPT rows) and key range, key tiles of 64 in two stages filled by
// asynchronous copies.  A thread owns RPT rows x 4 keys of S and RPT rows x 4
// dims of O; operands are read as 16-byte vectors along the summed dimension
// (row pitch 68 floats, so neighbouring rows start in different banks), which
// gives 16 RPT multiply-adds for RPT + 4 shared loads.  RPT = 2 up to 32 rows,
// else 4; 4 requests x 8 heads x 1000 rows over 512-2048 positions 313 us (26
// TFLOP/s; 430 with RPT = 2).
//
// f32_rows_kernel.  Blocks and single tokens (up to 16 rows per KV head):
// the cache is read once, straight into registers.  Eight lanes share a key,
// eight dims each, so a warp reads four whole rows per load; a lane's partial
// dot products of 8 rows are exchanged so that each lane ends up with one
// row's score (7 shuffles), takes its weight, and hands it back to the group
// for the value sum.  No barrier stands in the loop.  The key range is shared
// by a cluster of up to 8 CTAs, whose statistics and values meet through
// distributed shared memory; the scores wait in shared memory until the rows'
// log-sum-exp is known, so that each CTA adds its own positions' weights: one
// launch (8 requests x 6 heads x 16 rows over 112-448 positions with weights
// 16.4 us, a chain of latencies).  Longer ranges are split and joined by a
// second kernel.
//
// f32_mass_kernel.  The weights of a tile of 64 keys: the keys stay in shared
// memory, the rows pass by, each thread sums its rows of 4 keys, and the 16
// row groups are added in order at the end.
#include <algorithm>
#include <type_traits>

#include "ws_pattn.cuh"

namespace {

constexpr int TK = 64, NT = 256, PITCH = WS_DH + 4;
constexpr int MAT = TK * PITCH;                    // floats of a 64-row matrix

__device__ __forceinline__ void cp16(float* dst, const float* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows r0 .. of a unit as a [rows][PITCH] matrix, times the sign of scale
// (zero where scale is 0, or past R).
__device__ __forceinline__ void load_q(const AttnP& p, const Req& r, int h, int r0, int R, int rows, float* sq) {
  for (int x = threadIdx.x; x < rows * 16; x += NT) {
    const int row = x >> 4, c = x & 15, rho = r0 + row;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rho < R && p.a.scale != 0.f) {
      const int t = rho / p.G;
      v = __ldg(reinterpret_cast<const float4*>((const float*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride +
                                                (size_t)(h * p.G + rho - t * p.G) * WS_DH) + c);
      if (p.a.scale < 0.f) v = make_float4(-v.x, -v.y, -v.z, -v.w);
    }
    *reinterpret_cast<float4*>(sq + row * PITCH + 4 * c) = v;
  }
}
// 64 cache rows from position j0 on (zeros where there is none); returns
// whether this thread's key (thread < 64) counts.
__device__ __forceinline__ bool load_keys(const AttnP& p, const Req& r, int h, int j0, int limit, float* sk, float* sv) {
  bool valid = false;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int row = (threadIdx.x >> 4) + 16 * x, c = threadIdx.x & 15, pos = j0 + row;
    const int page = pos < limit ? paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, pos) : -1;
    const size_t off = page >= 0 ? paged_off(p.c, page, h, pos) + 4 * c : 0;
    cp16(sk + row * PITCH + 4 * c, (const float*)p.c.k + off, page >= 0);
    if (sv) cp16(sv + row * PITCH + 4 * c, (const float*)p.c.v + off, page >= 0);
  }
  if (threadIdx.x < TK) {
    const int pos = j0 + threadIdx.x;
    valid = pos < limit && paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, pos) >= 0;
  }
  return valid;
}

// s[a][b] = row (ty + 16 a) of A . row (tx + 16 b) of B over 64 columns
template <int RPT>
__device__ __forceinline__ void dots(const float* A, const float* Bm, int ty, int tx, float s[RPT][4]) {
  float2 acc[RPT][4];
#pragma unroll
  for (int a = 0; a < RPT; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < WS_DH; d += 4) {
    float4 q[RPT], k[4];
#pragma unroll
    for (int a = 0; a < RPT; ++a) q[a] = *reinterpret_cast<const float4*>(A + (ty + 16 * a) * PITCH + d);
#pragma unroll
    for (int b = 0; b < 4; ++b) k[b] = *reinterpret_cast<const float4*>(Bm + (tx + 16 * b) * PITCH + d);
#pragma unroll
    for (int a = 0; a < RPT; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        acc[a][b] = __ffma2_rn(make_float2(q[a].x, q[a].y), make_float2(k[b].x, k[b].y), acc[a][b]);
        acc[a][b] = __ffma2_rn(make_float2(q[a].z, q[a].w), make_float2(k[b].z, k[b].w), acc[a][b]);
      }
  }
#pragma unroll
  for (int a = 0; a < RPT; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) s[a][b] = acc[a][b].x + acc[a][b].y;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(local)), "r"(rank));
  return a;
}

// Weight of a part with maximum x (log2 units) beside one of M.  Parts that
// saw nothing are multiplied by 0, not left out: their sum is 0, or NaN where
// every score was, and a NaN has to reach the result.
__device__ __forceinline__ float weight_of(float x, float M) { return x == -INFINITY ? 0.f : ex2(x - M); }

// grid (cs, heads, requests), cluster (cs, 1, 1) where the CTAs join their
// parts themselves (JOIN), else the CTAs write split partials.
constexpr int CL_MAX = 8, CL_KEYS = 1024;           // CTAs per cluster, positions per CTA whose scores are kept
constexpr int RW = 4, RNT = RW * 32;                // warps
constexpr int rows_smem(int keys) { return (16 * PITCH + RW * 16 * PITCH + 16 * (keys + 4)) * 4; }

// NR rows per lane group: 8, or 2 for single tokens.
template <int NR, bool MASS, bool JOIN>
__global__ void __launch_bounds__(RNT, NR == 8 ? 3 : 4) f32_rows_kernel(const AttnP p, int cs, int keys) {
  constexpr int U = 4;                              // keys of a group in flight
  extern __shared__ __align__(16) float fsm[];
  __shared__ float2 wstat[RW][16];                  // a warp's (max, sum) per row
  __shared__ float2 stat[16];                       // this CTA's
  __shared__ float2 all[CL_MAX][16];
  __shared__ float row_lse[16];                     // log2 units, +inf for a row that sees nothing
  const int h = blockIdx.y, i = blockIdx.z, rank = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane >> 3, c = lane & 7;
  pdl_trigger();
  const Req r = request(p, i);
  const int R = r.c * p.G;
  if (R == 0) return;                               // the whole cluster leaves
  float *sq = fsm, *so = sq + 16 * PITCH, *stash = so + RW * 16 * PITCH;
  const int pitch = keys + 4;
  for (int x = threadIdx.x; x < 16 * 16; x += RNT) {
    const int row = x >> 4, d = x & 15;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < R && p.a.scale != 0.f) {
      const int t = row / p.G;
      v = __ldg(reinterpret_cast<const float4*>((const float*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride +
                                                (size_t)(h * p.G + row - t * p.G) * WS_DH) + d);
      if (p.a.scale < 0.f) v = make_float4(-v.x, -v.y, -v.z, -v.w);
    }
    *reinterpret_cast<float4*>(sq + row * PITCH + 4 * d) = v;
  }
  __syncthreads();
  // warps take row groups in turn and, within one, every KW-th step of four
  // keys; two warps for a group of a context's block, whose rows have to come
  // out the same bits in a block of any height
  const int RG = (R + NR - 1) / NR, KW = p.pad_H ? 2 : RG >= RW ? 1 : RW / RG, kw = warp / RG;
  // a cluster shares what the request has (64 requests x 6 heads x 16 rows
  // over 512-2048 positions with weights: 246 us with fixed ranges, 193 so);
  // split CTAs take fixed ranges and leave at once where there is nothing
  const int mine = JOIN ? min(keys, ((r.L + cs - 1) / cs + 3) & ~3) : keys;
  const int kb = min(r.L, rank * mine), ke = min(r.L, kb + mine);
  const int all_see = row_limit(p, r, 0);           // positions that every row sees
  const bool works = kw < KW;
  for (int rg = warp % RG; works && rg < RG; rg += RW) {
    const int row = rg * NR + (NR == 8 ? c : c & 1);   // the row whose score this lane ends up with
    const int lim = row < R ? min(ke, row_limit(p, r, row / p.G)) : 0;
    float m = -INFINITY, msl = 0.f, l = 0.f;
    float2 o[NR][4];
#pragma unroll
    for (int a = 0; a < NR; ++a)
#pragma unroll
      for (int d = 0; d < 4; ++d) o[a][d] = make_float2(0.f, 0.f);
    for (int j0 = kb + kw * 4 + grp; __any_sync(0xffffffffu, j0 < ke); j0 += U * KW * 4) {
      float4 k[U][2], v[U][2];
      uint32_t valid = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * KW * 4;
        const int page = j < ke ? paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, j) : -1;
        k[u][0] = k[u][1] = v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (page >= 0) {
          valid |= 1u << u;
          const size_t off = paged_off(p.c, page, h, j) + 8 * c;
          const float4* kp = reinterpret_cast<const float4*>((const float*)p.c.k + off);
          const float4* vp = reinterpret_cast<const float4*>((const float*)p.c.v + off);
          k[u][0] = __ldg(kp); k[u][1] = __ldg(kp + 1);
          v[u][0] = __ldg(vp); v[u][1] = __ldg(vp + 1);
        }
      }
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = 0.f;
      {
        float part[U][NR];
#pragma unroll
        for (int a = 0; a < NR; ++a) {
          const float4 qa = *reinterpret_cast<const float4*>(sq + (rg * NR + a) * PITCH + 8 * c);
          const float4 qb = *reinterpret_cast<const float4*>(sq + (rg * NR + a) * PITCH + 8 * c + 4);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float2 s = make_float2(0.f, 0.f);
            s = __ffma2_rn(make_float2(qa.x, qa.y), make_float2(k[u][0].x, k[u][0].y), s);
            s = __ffma2_rn(make_float2(qa.z, qa.w), make_float2(k[u][0].z, k[u][0].w), s);
            s = __ffma2_rn(make_float2(qb.x, qb.y), make_float2(k[u][1].x, k[u][1].y), s);
            s = __ffma2_rn(make_float2(qb.z, qb.w), make_float2(k[u][1].z, k[u][1].w), s);
            part[u][a] = s.x + s.y;
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (NR == 8) {
            float w4[4], w2[2];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const float give = c & 4 ? part[u][a] : part[u][(a + 4) % NR], keep = c & 4 ? part[u][(a + 4) % NR] : part[u][a];
              w4[a] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              const float give = c & 2 ? w4[a] : w4[a + 2], keep = c & 2 ? w4[a + 2] : w4[a];
              w2[a] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
            }
            const float give = c & 1 ? w2[0] : w2[1], keep = c & 1 ? w2[1] : w2[0];
            x[u] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
          } else {
            // lanes with c odd keep row 1, even row 0
            const float give = c & 1 ? part[u][0] : part[u][1], keep = c & 1 ? part[u][1] : part[u][0];
            float w = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            w += __shfl_xor_sync(0xffffffffu, w, 2);
            x[u] = w + __shfl_xor_sync(0xffffffffu, w, 4);
          }
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * KW * 4;
        if (!((valid >> u) & 1u) || j >= lim) x[u] = -INFINITY;
        if (MASS && j < ke && row < R && (NR == 8 || c < 2)) stash[row * pitch + j - kb] = x[u];
        top = fmaxf(top, x[u]);
      }
      // the reference moves only when a score passes it by more than 2^8
      const bool grow = top * p.sl > msl + 8.f || (m == -INFINITY && top > -INFINITY);
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? top : m;
        const float f = m > -INFINITY ? ex2((m - mn) * p.sl) : 0.f;
        m = mn;
        msl = mn > -INFINITY ? mn * p.sl : 0.f;
        l *= f;
#pragma unroll
        for (int a = 0; a < NR; ++a) {
          const float fa = __shfl_sync(0xffffffffu, f, a, 8);
#pragma unroll
          for (int d = 0; d < 4; ++d) { o[a][d].x *= fa; o[a][d].y *= fa; }
        }
      }
      // where some row does not see all of the keys, a weight of zero takes no
      // value: 0 * inf would reach the rows before an infinite one
      auto add_values = [&](auto mixed) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float e = ex2(fmaf(x[u], p.sl, -msl));
          l += e;
#pragma unroll
          for (int a = 0; a < NR; ++a) {
            const float w = __shfl_sync(0xffffffffu, e, a, 8);
            if (decltype(mixed)::value && w == 0.f) continue;
            const float2 w2 = make_float2(w, w);
            o[a][0] = __ffma2_rn(w2, make_float2(v[u][0].x, v[u][0].y), o[a][0]);
            o[a][1] = __ffma2_rn(w2, make_float2(v[u][0].z, v[u][0].w), o[a][1]);
            o[a][2] = __ffma2_rn(w2, make_float2(v[u][1].x, v[u][1].y), o[a][2]);
            o[a][3] = __ffma2_rn(w2, make_float2(v[u][1].z, v[u][1].w), o[a][3]);
          }
        }
      };
      if (all_see < ke && j0 - grp + (U - 1) * KW * 4 + 4 > all_see) add_values(std::true_type());
      else add_values(std::false_type());
    }
    // ---- the warp's four groups
    float M = m;
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
    const float f = m == -INFINITY ? 0.f : ex2((m - M) * p.sl);
    l *= f;
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
    for (int a = 0; a < NR; ++a) {
      const float fa = __shfl_sync(0xffffffffu, f, a, 8);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        float2 y = make_float2(o[a][d].x * fa, o[a][d].y * fa);
        y.x += __shfl_xor_sync(0xffffffffu, y.x, 8); y.y += __shfl_xor_sync(0xffffffffu, y.y, 8);
        y.x += __shfl_xor_sync(0xffffffffu, y.x, 16); y.y += __shfl_xor_sync(0xffffffffu, y.y, 16);
        if (grp == 0) *reinterpret_cast<float2*>(so + (kw * 16 + rg * NR + a) * PITCH + 8 * c + 2 * d) = y;
      }
    }
    if (grp == 0 && (NR == 8 || c < 2)) wstat[kw][row] = make_float2(M == -INFINITY ? M : M * p.sl, l);
  }
  __syncthreads();
  // ---- the CTA's warps: thread (row, 8 dims)
  {
    const int row = threadIdx.x >> 3, d = (threadIdx.x & 7) * 8;
    if (row < R) {
      float M = -INFINITY, sum = 0.f;
      for (int k = 0; k < KW; ++k) M = fmaxf(M, wstat[k][row].x);
      float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
      for (int k = 0; k < KW; ++k) {
        const float f = weight_of(wstat[k][row].x, M);
        sum = fmaf(f, wstat[k][row].y, sum);
        const float4 b0 = *reinterpret_cast<const float4*>(so + (k * 16 + row) * PITCH + d);
        const float4 b1 = *reinterpret_cast<const float4*>(so + (k * 16 + row) * PITCH + d + 4);
        a0.x = fmaf(f, b0.x, a0.x); a0.y = fmaf(f, b0.y, a0.y); a0.z = fmaf(f, b0.z, a0.z); a0.w = fmaf(f, b0.w, a0.w);
        a1.x = fmaf(f, b1.x, a1.x); a1.y = fmaf(f, b1.y, a1.y); a1.z = fmaf(f, b1.z, a1.z); a1.w = fmaf(f, b1.w, a1.w);
      }
      if (JOIN) {
        // into warp 0's area: read above by this thread alone
        *reinterpret_cast<float4*>(so + row * PITCH + d) = a0;
        *reinterpret_cast<float4*>(so + row * PITCH + d + 4) = a1;
        if (d == 0) stat[row] = make_float2(M, sum);
      } else {
        const size_t at = (((size_t)i * p.c.n_kv_heads + h) * ((size_t)p.a.max_q * p.G) + row) * p.nsplit + rank;
        *reinterpret_cast<float4*>(p.part_o + at * WS_DH + d) = a0;
        *reinterpret_cast<float4*>(p.part_o + at * WS_DH + d + 4) = a1;
        if (d == 0) p.part_ml[at] = make_float2(M, sum);
      }
    }
  }
  if (!JOIN) return;
  if (cs > 1) cluster_sync(); else __syncthreads();
  // ---- every CTA learns all statistics; each joins the values of its rows
  for (int x = threadIdx.x; x < 16 * cs; x += RNT) {
    const int k = x >> 4, row = x & 15;
    float2 y = make_float2(-INFINITY, 0.f);
    if (row < R) {
      if (cs > 1)
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(remote(&stat[row], (uint32_t)k)));
      else
        y = stat[row];
    }
    all[k][row] = y;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * 16; x += RNT) {
    const int row = x >> 4, d = (x & 15) * 4;
    float M = -INFINITY, sum = 0.f;
    for (int k = 0; k < cs; ++k) M = fmaxf(M, all[k][row].x);
    for (int k = 0; k < cs; ++k) sum = fmaf(weight_of(all[k][row].x, M), all[k][row].y, sum);
    if (d == 0) row_lse[row] = sum == 0.f ? INFINITY : M + lg2(sum);
    if (row % cs != rank) continue;
    float4 part[CL_MAX];
#pragma unroll
    for (int k = 0; k < CL_MAX; ++k) {
      part[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < cs) {
        if (cs > 1)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(part[k].x), "=f"(part[k].y), "=f"(part[k].z), "=f"(part[k].w)
                       : "r"(remote(so + row * PITCH + d, (uint32_t)k)));
        else
          part[k] = *reinterpret_cast<const float4*>(so + row * PITCH + d);
      }
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < CL_MAX; ++k)
      if (k < cs) {
        const float f = weight_of(all[k][row].x, M);
        a.x = fmaf(f, part[k].x, a.x); a.y = fmaf(f, part[k].y, a.y);
        a.z = fmaf(f, part[k].z, a.z); a.w = fmaf(f, part[k].w, a.w);
      }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = row / p.G, u = h * p.G + row - t * p.G;
    float* out = (float*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u * WS_DH + d;
    *reinterpret_cast<float4*>(out) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (p.lse && d == 0) p.lse[(size_t)(r.row0 + t) * p.a.n_heads + u] = sum == 0.f ? -INFINITY : (M + lg2(sum)) * LN2;
  }
  if (MASS) {
    __syncthreads();
    float* mass = p.a.mass + ((size_t)r.slot * p.c.n_kv_heads + h) * p.a.mass_stride;
    for (int x = threadIdx.x; x < ke - kb; x += RNT) {
      const int pos = kb + x;
      if (paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, pos) < 0) continue;
      float w = 0.f;
      for (int row = 0; row < R; ++row) {           // a NaN log-sum-exp adds NaN where its row sees, and nothing elsewhere
        const float y = stash[row * pitch + x];
        if (y != -INFINITY) w += ex2(fmaf(y, p.sl, -row_lse[row]));
      }
      atomicAdd(mass + pos, w);                     // this thread's position alone
    }
  }
  if (cs > 1) cluster_sync();                       // nobody leaves while its values are read
}

template <int RPT>
constexpr int f32_smem() { return (2 * 16 * RPT * PITCH + 4 * MAT) * 4; }   // Q, P, two stages of K and V

template <int RPT>
__global__ void __launch_bounds__(NT, 2) f32_kernel(const AttnP p) {
  extern __shared__ __align__(16) float fsm[];
  __shared__ uint32_t s_valid[2][2];
  const int rt = blockIdx.x / p.nsplit, split = blockIdx.x - rt * p.nsplit, h = blockIdx.y, i = blockIdx.z;
  pdl_trigger();
  const Req r = request(p, i);
  constexpr int TQ = 16 * RPT;
  const int R = r.c * p.G, r0 = rt * TQ;
  if (r0 >= R) return;
  float *sq = fsm, *sp = sq + TQ * PITCH, *stage = sp + TQ * PITCH;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int last = min(R, r0 + TQ) - 1, Lmax = row_limit(p, r, last / p.G), Lmin = row_limit(p, r, r0 / p.G);
  const int nt = (Lmax + TK - 1) / TK, tb = min(nt, split * p.tps), te = min(nt, tb + p.tps);
  auto fetch = [&](int t) {
    float* k = stage + (t & 1) * 2 * MAT;
    const bool v = load_keys(p, r, h, t * TK, Lmax, k, k + MAT);
    const uint32_t b = __ballot_sync(0xffffffffu, v);
    if (threadIdx.x < TK && (threadIdx.x & 31) == 0) s_valid[t & 1][threadIdx.x >> 5] = b;
    cp_commit();
  };
  if (tb < te) fetch(tb);
  load_q(p, r, h, r0, R, TQ, sq);
  int lim[RPT];
  float m[RPT], l[RPT];
  float2 o[RPT][2];
#pragma unroll
  for (int a = 0; a < RPT; ++a) {
    lim[a] = row_limit(p, r, min(r0 + ty + 16 * a, R - 1) / p.G);
    m[a] = -INFINITY;
    l[a] = 0.f;
    o[a][0] = o[a][1] = make_float2(0.f, 0.f);
  }
  for (int t = tb; t < te; ++t) {
    if (t + 1 < te) { fetch(t + 1); cp_wait<1>(); } else cp_wait<0>();
    __syncthreads();
    const float* k = stage + (t & 1) * 2 * MAT;
    const float* v = k + MAT;
    float s[RPT][4];
    dots<RPT>(sq, k, ty, tx, s);
    const uint32_t v0 = s_valid[t & 1][0], v1 = s_valid[t & 1][1];
    if ((v0 & v1) != 0xffffffffu || (t + 1) * TK > Lmin) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int j = tx + 16 * b;
        const bool ok = ((b < 2 ? v0 : v1) >> (j & 31)) & 1u;
#pragma unroll
        for (int a = 0; a < RPT; ++a)
          if (!ok || t * TK + j >= lim[a]) s[a][b] = -INFINITY;
      }
    }
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      float mx = fmaxf(fmaxf(s[a][0], s[a][1]), fmaxf(s[a][2], s[a][3]));
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[a], mx * p.sl);     // statistics in log2 units
      const float f = m[a] == -INFINITY ? 0.f : ex2(m[a] - mn), ref = mn == -INFINITY ? 0.f : mn;
      m[a] = mn;
      l[a] *= f;
      o[a][0].x *= f; o[a][0].y *= f; o[a][1].x *= f; o[a][1].y *= f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float e = ex2(fmaf(s[a][b], p.sl, -ref));
        l[a] += e;
        sp[(ty + 16 * a) * PITCH + tx + 16 * b] = e;
      }
    }
    __syncwarp();                                  // a row of P is written and read by one half-warp
    // where some row does not see all of the keys, a weight of zero takes no
    // value: 0 * inf would reach the rows before an infinite one
    auto add_values = [&](auto mixed) {
#pragma unroll 4
      for (int j = 0; j < TK; j += 4) {
        float4 w[RPT], x[4];
#pragma unroll
        for (int a = 0; a < RPT; ++a) w[a] = *reinterpret_cast<const float4*>(sp + (ty + 16 * a) * PITCH + j);
#pragma unroll
        for (int b = 0; b < 4; ++b) x[b] = *reinterpret_cast<const float4*>(v + (j + b) * PITCH + 4 * tx);
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
          const float ws[4] = {w[a].x, w[a].y, w[a].z, w[a].w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (decltype(mixed)::value && ws[b] == 0.f) continue;
            const float2 w2 = make_float2(ws[b], ws[b]);
            o[a][0] = __ffma2_rn(w2, make_float2(x[b].x, x[b].y), o[a][0]);
            o[a][1] = __ffma2_rn(w2, make_float2(x[b].z, x[b].w), o[a][1]);
          }
        }
      }
    };
    if (Lmin < Lmax && (t + 1) * TK > Lmin) add_values(std::true_type());
    else add_values(std::false_type());
    __syncthreads();                               // the stage and P are free
  }
#pragma unroll
  for (int a = 0; a < RPT; ++a) {
    const int rho = r0 + ty + 16 * a;
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], x);
    if (rho >= R) continue;
    if (p.nsplit > 1) {
      const size_t at = (((size_t)i * p.c.n_kv_heads + h) * ((size_t)p.a.max_q * p.G) + rho) * p.nsplit + split;
      *reinterpret_cast<float4*>(p.part_o + at * WS_DH + 4 * tx) = make_float4(o[a][0].x, o[a][0].y, o[a][1].x, o[a][1].y);
      if (tx == 0) p.part_ml[at] = make_float2(m[a], l[a]);
      continue;
    }
    const int t = rho / p.G, u = h * p.G + rho - t * p.G;
    const float inv = l[a] == 0.f ? 0.f : 1.f / l[a];
    float* out = (float*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u * WS_DH + 4 * tx;
    *reinterpret_cast<float4*>(out) = make_float4(o[a][0].x * inv, o[a][0].y * inv, o[a][1].x * inv, o[a][1].y * inv);
    if (p.lse && tx == 0) p.lse[(size_t)(r.row0 + t) * p.a.n_heads + u] = l[a] == 0.f ? -INFINITY : (m[a] + lg2(l[a])) * LN2;
  }
}

template <int RPT>
constexpr int mass_smem() { return (16 * RPT * PITCH + MAT) * 4; }

template <int RPT>
__global__ void __launch_bounds__(NT, 2) f32_mass_kernel(const AttnP p) {
  extern __shared__ __align__(16) float fsm[];
  __shared__ float part[16][TK];
  constexpr int TQ = 16 * RPT;
  const int h = blockIdx.y, i = blockIdx.z, j0 = blockIdx.x * TK;
  const Req r = request(p, i);
  if (j0 >= r.L || r.c == 0) {                     // waits all the same: this grid's end has to follow the rows' kernels'
    pdl_wait();
    return;
  }
  float *sq = fsm, *sk = sq + TQ * PITCH;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, R = r.c * p.G;
  const bool valid = load_keys(p, r, h, j0, r.L, sk, nullptr);
  cp_commit();
  pdl_wait();                                      // the log-sum-exps
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  // rows before the first that sees position j0 add nothing
  for (int r0 = p.a.causal ? max(0, j0 - (r.L - r.c)) * p.G : 0; r0 < R; r0 += TQ) {
    __syncthreads();
    load_q(p, r, h, r0, R, TQ, sq);
    cp_wait<0>();
    __syncthreads();
    float s[RPT][4];
    dots<RPT>(sq, sk, ty, tx, s);
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      const int rho = r0 + ty + 16 * a;
      if (rho >= R) continue;
      const int t = rho / p.G, lim = row_limit(p, r, t);
      const float x = p.lse[(size_t)(r.row0 + t) * p.a.n_heads + h * p.G + rho - t * p.G];
      if (x == -INFINITY) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (j0 + tx + 16 * b < lim) sum[b] += ex2(fmaf(s[a][b], p.sl, -x * LOG2E));
    }
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) part[ty][tx + 16 * b] = sum[b];
  __syncthreads();
  if (threadIdx.x < TK && valid) {
    float total = 0.f;
#pragma unroll
    for (int x = 0; x < 16; ++x) total += part[x][threadIdx.x];
    p.a.mass[((size_t)r.slot * p.c.n_kv_heads + h) * p.a.mass_stride + j0 + threadIdx.x] += total;
  }
}

template <int RPT>
cudaError_t run_f32(const AttnP& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(f32_kernel<RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, f32_smem<RPT>());
  if (e != cudaSuccess) return e;
  f32_kernel<RPT><<<dim3(p.row_tiles * p.nsplit, p.c.n_kv_heads, p.a.n_req), NT, f32_smem<RPT>(), s>>>(p);
  ws_count_launches(1);
  return cudaGetLastError();
}
template <int RPT>
cudaError_t run_mass(const AttnP& p, cudaStream_t s) {
  return launch_after(f32_mass_kernel<RPT>, dim3((p.a.max_kv + TK - 1) / TK, p.c.n_kv_heads, p.a.n_req), NT,
                      mass_smem<RPT>(), s, p);
}

}  // namespace

template <int NR, bool MASS, bool JOIN>
static cudaError_t run_rows(const AttnP& p, int cs, int keys, cudaStream_t s) {
  const auto kern = f32_rows_kernel<NR, MASS, JOIN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem(MASS ? CL_KEYS : 0));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(cs, p.c.n_kv_heads, p.a.n_req);
  c.blockDim = dim3(RNT);
  c.dynamicSmemBytes = rows_smem(MASS ? keys : 0);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = JOIN ? (unsigned)cs : 1u; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, kern, p, cs, keys);
  if (e == cudaSuccess) ws_count_launches(1);
  return e;
}

cudaError_t launch_f32_rows(const AttnP& p, const F32Rows& f, cudaStream_t s) {
  // one or two rows: 8 requests x 6 heads x 448 positions 20 us, 24 with groups of eight rows
  // (a context's block keeps the larger groups: their sums run in another order)
  const bool one = (long long)p.a.max_q * p.G <= 2 && !p.pad_H, mass = p.a.mass != nullptr;
  if (!f.join) return one ? run_rows<2, false, false>(p, f.ctas, f.keys, s) : run_rows<8, false, false>(p, f.ctas, f.keys, s);
  if (mass) return one ? run_rows<2, true, true>(p, f.ctas, f.keys, s) : run_rows<8, true, true>(p, f.ctas, f.keys, s);
  return one ? run_rows<2, false, true>(p, f.ctas, f.keys, s) : run_rows<8, false, true>(p, f.ctas, f.keys, s);
}

F32Rows f32_rows_plan(long long units, int max_kv, bool mass) {
  // About three rounds of three CTAs per SM; none shorter than 64 positions,
  // and none shorter than 256 beyond the first round (64 requests x 6 heads x
  // 16 rows over 112-448 positions: seven CTAs each 87 us, one each 62).
  constexpr long long ROUND = 3 * 152;
  long long want = (3 * ROUND + units - 1) / units;
  want = std::min(want, std::max({ROUND / units, max_kv / 256ll, 1ll}));
  want = std::min(want, std::max(max_kv / 64ll, 1ll));
  F32Rows f;
  // One launch where a cluster's CTAs are enough, and keep their scores.
  // Without weights and beyond one round a second kernel joins faster, because
  // nothing waits for the cluster's last CTA (16 rows over 512-2048 positions:
  // 24 requests 80 us against 97, 64 requests 168 against 179; 8 requests, one
  // round, 448 positions: 27 against 30).
  const bool fits = !mass || max_kv <= CL_MAX * CL_KEYS;
  f.join = fits && (mass || units * want <= ROUND) && (want <= CL_MAX || max_kv <= CL_MAX * 512);
  if (f.join && want > CL_MAX) want = CL_MAX;
  if (f.join && mass && want * CL_KEYS < max_kv) want = (max_kv + CL_KEYS - 1) / CL_KEYS;
  f.keys = (int)(((max_kv > 0 ? max_kv : 1) + want - 1) / want);
  f.keys = (f.keys + 3) / 4 * 4;
  f.ctas = ((max_kv > 0 ? max_kv : 1) + f.keys - 1) / f.keys;
  return f;
}

F32Rows f32_block_plan(int max_kv) {
  F32Rows f;
  f.join = true;
  const int want = std::max(1, std::min(CL_MAX, max_kv / 256));
  f.keys = ((std::max(max_kv, 1) + want - 1) / want + 3) / 4 * 4;
  f.ctas = (std::max(max_kv, 1) + f.keys - 1) / f.keys;
  return f;
}

cudaError_t launch_f32(const AttnP& p, int rpt, cudaStream_t s) { return rpt == 2 ? run_f32<2>(p, s) : run_f32<4>(p, s); }
cudaError_t launch_f32_mass(const AttnP& p, int rpt, cudaStream_t s) {
  return rpt == 0 ? run_mass<1>(p, s) : rpt == 2 ? run_mass<2>(p, s) : run_mass<4>(p, s);
}

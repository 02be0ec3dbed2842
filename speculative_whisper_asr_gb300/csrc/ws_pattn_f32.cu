// ws_paged_attention for the fp32 model: everything in fp32 on the FMA pipes
// (the tensor cores have no fp32 product).
//
// f32_kernel.  One CTA of 256 threads per (request, KV head, row tile of
// 16 * RPT rows) and key range, key tiles of 64 in two stages filled by
// asynchronous copies.  A thread owns RPT rows x 4 keys of S and RPT rows x 4
// dims of O; operands are read as 16-byte vectors along the summed dimension
// (row pitch 68 floats, so neighbouring rows start in different banks), which
// gives 16 RPT multiply-adds for RPT + 4 shared loads.  RPT = 4 is bound by
// the FMA pipe; RPT = 1 (16 rows: blocks and single tokens) by latency, so
// its key range is cut into as many splits as fill the machine.
//
// f32_mass_kernel.  The weights of a tile of 64 keys: the keys stay in shared
// memory, the rows pass by, each thread sums its rows of 4 keys, and the 16
// row groups are added in order at the end.
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
          const float2 w2 = make_float2(ws[b], ws[b]);
          o[a][0] = __ffma2_rn(w2, make_float2(x[b].x, x[b].y), o[a][0]);
          o[a][1] = __ffma2_rn(w2, make_float2(x[b].z, x[b].w), o[a][1]);
        }
      }
    }
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
  if (j0 >= r.L || r.c == 0) return;
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

cudaError_t launch_f32(const AttnP& p, bool wide, cudaStream_t s) { return wide ? run_f32<4>(p, s) : run_f32<1>(p, s); }
cudaError_t launch_f32_mass(const AttnP& p, bool wide, cudaStream_t s) { return wide ? run_mass<4>(p, s) : run_mass<1>(p, s); }

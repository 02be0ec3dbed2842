// Appending keys and values to a paged cache, with the position rotation of
// keys and queries on the way (ws_cache_append in include/ws.h gives the
// formulas).
//
// A CTA takes a tile of consecutive tokens of one request (in a cache in 8
// bits one block of one scale, or 64 tokens of a longer one) and some of the
// heads; a warp takes a head of queries, keys or values at a time: lane l
// holds elements of token l / 8 + 4 j, so a warp's access covers whole rows.
// The cosines and sines are computed once per tile into shared memory and
// serve all its heads.  An angle is the 64-bit product of the position and
// the turns per position, whose overflow drops whole turns exactly; its top 32
// bits, as a fraction of half a turn, go through sincospif.  The rows are
// asked for as soon as the chunk's place in them is known, before the angles.
// In 8 bits the lanes find the block's largest value first (the rows stay in
// registers), which gives the scale's exponent from the bits of the maximum;
// then the elements are multiplied by a power of two (exact) and rounded
// once.  Only where an older block's scale grows are its earlier tokens read.
#include <string>

#include "ws_paged.cuh"

namespace {

constexpr int AP_W = 8;                    // warps
constexpr int AP_T = 64;                   // tokens at a time, at most

struct AppendP {
  ws_paged_cache c;
  ws_append_args a;
  int items;                               // heads of queries, keys and values
  int tile;                                // tokens per CTA
};

__device__ __forceinline__ float pow2(int k) {           // 2^k, k in -254 .. 127, as far as fp32 reaches
  return k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23) : k >= -149 ? __uint_as_float(1u << (k + 149)) : 0.f;
}
// Exponent of the smallest power of two s with m <= 448 s = 1.75 * 2^8 s (m finite, >= 0).
__device__ __forceinline__ int scale_exponent(float m) {
  const uint32_t u = __float_as_uint(m);
  return max(-127, (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3_pair(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  float2 f;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// Eight elements of a row: four from o1 on and four from o2 on.
struct Piece { int o1, o2, pair; bool turns; };           // the pairs (o1 + 0, + 1), ... or (o1 + e, o2 + e) are pair, pair + 1, ...
template <class T> struct Raw;
template <> struct Raw<bf16> { uint2 a, b; };
template <> struct Raw<float> { float4 a, b; };

template <class T>
__device__ __forceinline__ void load_piece(const T* row, const Piece& pc, Raw<T>& r) {
  using V = decltype(r.a);
  r.a = *reinterpret_cast<const V*>(row + pc.o1);
  r.b = *reinterpret_cast<const V*>(row + pc.o2);
}
__device__ __forceinline__ float2 two(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }
__device__ __forceinline__ void unpack(const Raw<bf16>& r, float* x) {
  const float2 p = two(r.a.x), q = two(r.a.y), s = two(r.b.x), t = two(r.b.y);
  x[0] = p.x; x[1] = p.y; x[2] = q.x; x[3] = q.y; x[4] = s.x; x[5] = s.y; x[6] = t.x; x[7] = t.y;
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float* x) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w; x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store_piece(bf16* row, const Piece& pc, const float* x) {
  *reinterpret_cast<uint2*>(row + pc.o1) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  *reinterpret_cast<uint2*>(row + pc.o2) = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store_piece(float* row, const Piece& pc, const float* x) {
  *reinterpret_cast<float4*>(row + pc.o1) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(row + pc.o2) = make_float4(x[4], x[5], x[6], x[7]);
}
// The rotation of a piece; cs: cosines of its four pairs, then (AP_T * 32 floats on) their sines.
__device__ __forceinline__ void turn(float* x, const float* cs, bool halves) {
  const float4 c4 = *reinterpret_cast<const float4*>(cs), s4 = *reinterpret_cast<const float4*>(cs + AP_T * 32);
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
  float y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p = halves ? x[e] : x[2 * e], q = halves ? x[4 + e] : x[2 * e + 1];
    const float u = p * c[e] - q * s[e], v = p * s[e] + q * c[e];
    if (halves) { y[e] = u; y[4 + e] = v; } else { y[2 * e] = u; y[2 * e + 1] = v; }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = y[e];
}

// NP pieces per lane: tiles of up to 4 * NP tokens at a time.
template <class T, bool Q8, int NP>
__global__ void __launch_bounds__(AP_W * 32, 2) append_kernel(const AppendP p) {
  __shared__ __align__(16) float cs[2 * AP_T * 32];        // cosines, sines [token][pair]
  __shared__ int page_of[AP_T];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = blockIdx.z;
  const int slot = p.a.req_ids ? p.a.req_ids[i] : i;
  const int row0 = p.a.cu_q[i];
  const int c = row0 >= 0 ? min(max(min(p.a.cu_q[i + 1], p.a.total_q) - row0, 0), p.a.max_q) : 0;
  if (slot < 0 || slot >= p.c.n_slots || c == 0) return;
  const int L = p.a.kv_len[slot];
  const long long start = (long long)L - c;                // position of the chunk's first row
  if (L <= 0) return;
  // tokens lo .. hi - 1 of this CTA
  const int begin = (int)max(start, 0ll);
  const long long t0 = Q8 ? ((long long)(begin / p.tile) + blockIdx.x) * p.tile : start + (long long)blockIdx.x * p.tile;
  const int lo = (int)max(t0, (long long)begin), hi = (int)min(t0 + p.tile, (long long)L);
  if (lo >= hi) return;
  const bool halves = p.a.rot_halves != 0;
  const int nq = p.a.q ? p.a.n_heads : 0, nk = p.c.n_kv_heads;
  const int pairs = p.a.turns ? p.a.rot_dims / 2 : 0;
  Piece pc;
  {
    const int a = lane & 7;
    pc.turns = 8 * a < 2 * pairs;
    pc.pair = 4 * a;
    pc.o1 = halves && pc.turns ? 4 * a : 8 * a;
    pc.o2 = halves && pc.turns ? pairs + 4 * a : 8 * a + 4;
  }
  // a tile longer than AP_T tokens (a long block of one scale) is gone through
  // twice: for its largest values, then for its codes
  const bool whole = !Q8 || p.tile <= 4 * NP;
  __shared__ float s_max[Q8 ? 2 * 128 : 1];                // by key / value head of this CTA (long blocks)
  const int first_item = blockIdx.y * AP_W + warp, step = gridDim.y * AP_W;
  for (int pass = whole ? 1 : 0; pass < 2; ++pass)
    for (long long sub = Q8 ? (lo - t0) / (4 * NP) * (4 * NP) : 0; sub < p.tile && t0 + sub < hi; sub += 4 * NP) {
      const int base = (int)(t0 + sub);                    // first token of the visit (may lie before position 0)
      const int from = max(lo, base), to = (int)min((long long)hi, (long long)base + 4 * NP);
      __syncthreads();                                     // the last visit's angles have been read
      Raw<T> raw[NP];
      auto load = [&](int item) {
        const bool isq = item < nq, isk = !isq && item < nq + nk;
        const T* src = isq ? (const T*)p.a.q + (size_t)item * WS_DH
                           : isk ? (const T*)p.a.k + (size_t)(item - nq) * WS_DH : (const T*)p.a.v + (size_t)(item - nq - nk) * WS_DH;
        const int64_t ld = isq ? p.a.q_stride : isk ? p.a.k_stride : p.a.v_stride;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const int t = base + 4 * j + (lane >> 3);
          if (t >= from && t < to) load_piece(src + (size_t)(row0 + (t - start)) * ld, pc, raw[j]);
          else raw[j] = Raw<T>{};
        }
      };
      if (first_item < p.items) load(first_item);          // under the angles
      for (int x = tid; x < (to - from) * pairs; x += AP_W * 32) {
        const int t = x / pairs, f = x - t * pairs;
        const int m = p.a.pos ? p.a.pos[row0 + (from + t - start)] : from + t;
        const uint64_t phase = (uint64_t)(int64_t)m * p.a.turns[f];
        float s_, c_;
        sincospif((float)(int32_t)(uint32_t)(phase >> 32) * (1.f / 2147483648.f), &s_, &c_);
        cs[(from - base + t) * 32 + f] = c_;
        cs[AP_T * 32 + (from - base + t) * 32 + f] = s_;
      }
      for (int x = tid; x < to - from; x += AP_W * 32)
        page_of[from - base + x] = paged_page(p.c, p.c.page_table, p.c.table_stride, slot, from + x);
      __syncthreads();
      for (int item = first_item, n = 0; item < p.items; item += step, ++n) {
        if (n) load(item);
        const bool isq = item < nq, isk = !isq && item < nq + nk;
        const bool turned = pc.turns && (isq || isk);
        auto values = [&](int j, float* x) {
          unpack(raw[j], x);
          if (turned) turn(x, cs + (4 * j + (lane >> 3)) * 32 + pc.pair, halves);
        };
        if (isq) {
          if (pass == 0) continue;
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const int t = base + 4 * j + (lane >> 3);
            if (t < from || t >= to) continue;
            float x[8];
            values(j, x);
            store_piece((T*)p.a.q_out + (size_t)(row0 + (t - start)) * p.a.q_out_stride + (size_t)item * WS_DH, pc, x);
          }
          continue;
        }
        const int h = isk ? item - nq : item - nq - nk;
        if (!Q8) {
          T* dst = (T*)(isk ? p.c.k : p.c.v);
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const int t = base + 4 * j + (lane >> 3);
            if (t < from || t >= to) continue;
            const int page = page_of[t - base];
            if (page < 0) continue;
            float x[8];
            values(j, x);
            store_piece(dst + paged_off(p.c, page, h, t), pc, x);
          }
          continue;
        }
        // ---- 8 bits.  A block lies in one page.
        const int page = page_of[from - base];
        if (page < 0) continue;
        uint8_t* dst = (uint8_t*)(isk ? p.c.k : p.c.v) + paged_off(p.c, page, h, (int)t0);
        uint8_t* scale = (isk ? p.c.k_scale : p.c.v_scale) + scale_off(p.c, page, h, (int)t0);
        const bool begins = t0 >= begin;                   // with this call
        const int e_was = begins ? -127 : (int)*scale - 127;
        float m = 0.f;
        bool odd = false;
        if (whole || pass == 0) {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            float x[8];
            values(j, x);                                  // rows that are not there are zero
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float y = fabsf(x[e]);
              odd |= !(y < INFINITY);
              m = fmaxf(m, y < INFINITY ? y : 0.f);
            }
          }
#pragma unroll
          for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
          odd = __any_sync(0xffffffffu, odd);
          if (!whole) {
            if (lane == 0) s_max[n * AP_W + warp] = from == lo ? m : fmaxf(s_max[n * AP_W + warp], m);
            __syncwarp();
            continue;
          }
        } else {
          m = s_max[n * AP_W + warp];
          odd = true;
        }
        const int e_now = max(e_was, scale_exponent(m));
        const float f = pow2(-e_now);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const int t = base + 4 * j + (lane >> 3);
          if (t < from || t >= to) continue;
          float x[8];
          values(j, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = x[e] * f;
            x[e] = odd && !(fabsf(x[e]) < INFINITY) ? NAN : y;
          }
          uint8_t* at = dst + (size_t)(t - (int)t0) * (size_t)p.c.token_stride;
          *reinterpret_cast<uint32_t*>(at + pc.o1) = e4m3_pair(x[0], x[1]) | e4m3_pair(x[2], x[3]) << 16;
          *reinterpret_cast<uint32_t*>(at + pc.o2) = e4m3_pair(x[4], x[5]) | e4m3_pair(x[6], x[7]) << 16;
        }
        if (from != lo) continue;                          // once per block and head
        if (!begins && e_now > e_was) {                    // move the earlier tokens to the new scale
          const int down = e_was - e_now, half = down / 2;
          const float f1 = pow2(half), f2 = pow2(down - half);
          for (int x = lane; x < (begin - (int)t0) * 4; x += 32) {
            uint4* at = reinterpret_cast<uint4*>(dst + (size_t)(x >> 2) * (size_t)p.c.token_stride) + (x & 3);
            uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 a = from_e4m3_pair(w[e] & 0xFFFFu), b = from_e4m3_pair(w[e] >> 16);
              w[e] = e4m3_pair(a.x * f1 * f2, a.y * f1 * f2) | e4m3_pair(b.x * f1 * f2, b.y * f1 * f2) << 16;
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();                                      // every lane has read the old scale
        if (lane == 0 && (begins || e_now > e_was)) *scale = (uint8_t)(e_now + 127);
      }
    }
}

const char* check_append(const ws_paged_cache* c, const ws_append_args* a) {
  if (const char* e = check_paged_cache(c)) return e;
  if (!a) return "null arguments";
  if (a->n_req < 0 || a->n_req > 65535) return "n_req must be 0..65535";
  if (a->total_q < 0 || a->max_q < 0) return "negative size";
  if (a->max_q > 1 << 28) return "max_q must be at most 2^28";
  if (a->q && (a->n_heads < 1 || a->n_heads > 65535)) return "n_heads must be 1..65535";
  if (a->turns && (a->rot_dims < 8 || a->rot_dims > WS_DH || a->rot_dims % 8)) return "rot_dims must be a multiple of 8, 8..64";
  if (a->rot_halves != 0 && a->rot_halves != 1) return "rot_halves must be 0 or 1";
  if (a->n_req == 0 || a->total_q == 0) return nullptr;
  if (!a->kv_len || !a->cu_q || !a->k || !a->v) return "null kv_len, cu_q, k or v";
  if (a->q && !a->q_out) return "q without q_out";
  if (!a->q && a->q_out) return "q_out without q";
  const int64_t unit = 16 / row_es(*c), most = (int64_t)1 << 37;
  struct Rows { const void* p; int64_t stride; int64_t heads; };
  const Rows rows[4] = {{a->k, a->k_stride, c->n_kv_heads}, {a->v, a->v_stride, c->n_kv_heads},
                        {a->q, a->q_stride, a->n_heads}, {a->q_out, a->q_out_stride, a->n_heads}};
  for (const Rows& r : rows) {
    if (!r.p) continue;
    if ((reinterpret_cast<uintptr_t>(r.p) & 15) || r.stride % unit) return "rows of k, v, q and q_out must be 16-byte aligned";
    if (r.stride < r.heads * WS_DH) return "row strides must be >= 64 * heads";
    if (r.stride >= most) return "row stride too large";
  }
  if (a->turns && (reinterpret_cast<uintptr_t>(a->turns) & 7)) return "turns must be 8-byte aligned";
  if (!a->req_ids && a->n_req > c->n_slots) return "more requests than slots";
  const int64_t es = row_es(*c);
  if (a->q) {
    const int64_t qs = a->q_stride * es, os = a->q_out_stride * es, qw = (int64_t)a->n_heads * WS_DH * es,
                  kw = (int64_t)c->n_kv_heads * WS_DH * es;
    if (a->q == a->q_out ? qs != os && a->total_q > 1 : rows_overlap(a->q, qs, a->q_out, os, a->total_q, qw))
      return "q_out must be q with its stride, or share no elements with it";
    for (int x = 0; x < 2; ++x) {          // rows beside each other in one buffer are fine
      const char *o = (const char*)a->q_out, *r = (const char*)rows[x].p;
      const int64_t rs = rows[x].stride * es, n = a->total_q - 1;
      if (o >= r + n * rs + kw || r >= o + n * os + qw) continue;
      if (rs != os) return "q_out must share no elements with k and v";
      const int64_t d = ((o - r) % rs + rs) % rs;          // from a row of k or v on to a row of q_out
      if (d < kw || d + qw > rs) return "q_out must share no elements with k and v";
    }
  }
  return nullptr;
}

template <class T, bool Q8, int NP>
cudaError_t launch(const AppendP& p, dim3 grid, cudaStream_t s) {
  append_kernel<T, Q8, NP><<<grid, AP_W * 32, 0, s>>>(p);
  ws_count_launches(1);
  return cudaGetLastError();
}
template <class T, bool Q8>
cudaError_t launch_np(const AppendP& p, dim3 grid, cudaStream_t s) {
  if (p.tile <= 4) return launch<T, Q8, 1>(p, grid, s);
  if (p.tile <= 8) return launch<T, Q8, 2>(p, grid, s);
  if constexpr (Q8) {
    if (p.tile > 32) return launch<T, Q8, 16>(p, grid, s);
    if (p.tile > 16) return launch<T, Q8, 8>(p, grid, s);
  }
  return launch<T, Q8, 4>(p, grid, s);
}

}  // namespace

extern "C" int ws_cache_append(const ws_paged_cache* cache, const ws_append_args* args, ws_stream stream) {
  if (const char* e = check_append(cache, args)) return paged_fail(WS_EINVAL, e);
  if (args->n_req == 0 || args->total_q == 0 || args->max_q == 0) return WS_OK;
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  AppendP p = {};
  p.c = *cache;
  p.a = *args;
  const bool q8 = cache->dtype == WS_E4M3;
  p.items = (args->q ? args->n_heads : 0) + 2 * cache->n_kv_heads;
  p.tile = q8 ? cache->scale_block : args->max_q <= 4 ? 4 : args->max_q <= 8 ? 8 : 16;
  const long long tiles = q8 ? ((long long)args->max_q + p.tile - 2) / p.tile + 1 : (args->max_q + p.tile - 1) / p.tile;
  // a warp takes one head where there are few tiles; else as many as leave four CTAs per SM
  const int most = (p.items + AP_W - 1) / AP_W;
  const long long units = tiles * args->n_req;
  int groups = (int)min((long long)most, max(1ll, (4ll * 152 + units - 1) / units));
  // heads of a long block whose largest values a CTA keeps: 32 per warp
  if (q8) groups = max(groups, (p.items + 32 * AP_W - 1) / (32 * AP_W));
  if (tiles > 2147483647ll || groups > 65535) return paged_fail(WS_EINVAL, "too many tiles or heads");
  const dim3 grid((unsigned)tiles, (unsigned)groups, (unsigned)args->n_req);
  const cudaError_t e = q8 ? launch_np<bf16, true>(p, grid, (cudaStream_t)stream)
                           : cache->dtype == WS_BF16 ? launch_np<bf16, false>(p, grid, (cudaStream_t)stream)
                                                     : launch_np<float, false>(p, grid, (cudaStream_t)stream);
  if (e != cudaSuccess) return paged_fail(WS_ECUDA, std::string("cache append launch: ") + cudaGetErrorString(e));
  return WS_OK;
}

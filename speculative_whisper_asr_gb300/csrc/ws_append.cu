// Appending keys and values to a paged cache, with the position rotation of
// keys and queries on the way (ws_cache_append in include/ws.h gives the
// formulas).
//
// A CTA takes a tile of up to 64 consecutive tokens of one request (in a cache
// in 8 bits the tokens of one scale) and some of the heads.  A thread holds the
// same eight elements of the same token in every head, so the cosines and
// sines of its pairs are computed once, into registers.  An angle is the
// 64-bit product of the position and the turns per position, whose overflow
// drops whole turns exactly; its top 32 bits, as a fraction of half a turn, go
// through sincospif.  Heads are taken AP_H at a time, the next ones' rows under
// way meanwhile.  In 8 bits the CTA agrees on a head's largest value (as bits,
// so that what is not finite shows), which gives the scale's exponent; then
// the elements, still in registers, are multiplied by a power of two (exact)
// and rounded once.  A block of more than 64 tokens is gone through twice, for
// its largest values and for its codes.
// 4 chunks of up to 2048 rows, 32 query and 8 key/value heads in 8 bits (77 MB):
// 24.6 us, 3.1 TB/s; the copy rate would take 11.  What is left is latency: a
// tile's chain of lengths, page and rows, and the agreement on the scales.  (The
// 8-bit form spills four bytes at the 64 registers that let two CTAs of 512
// threads run on an SM.)
#include <string>
#include <type_traits>

#include "ws_paged.cuh"

namespace {

constexpr int AP_T = 64;                   // tokens at a time, at most: eight threads each
constexpr int AP_H = 2;                    // heads at a time (4, one CTA of 512 threads per SM: 29 us for 24.6)
constexpr int AP_MAX = 256;                // heads of a CTA, at most

struct AppendP {
  ws_paged_cache c;
  ws_append_args a;
  int items;                               // heads of queries, keys and values
  int per;                                 // of them per CTA
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

// Eight elements of a row: four from o1 on and four from o2 on, which lie
// together unless pairs are halves of the head.
struct Piece { int o1, o2; bool together, turns; };
template <class T> struct Raw;
template <> struct Raw<bf16> { uint2 a, b; };
template <> struct Raw<float> { float4 a, b; };

__device__ __forceinline__ void load_piece(const bf16* row, const Piece& pc, Raw<bf16>& r) {
  if (pc.together) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + pc.o1);
    r.a = make_uint2(v.x, v.y);
    r.b = make_uint2(v.z, v.w);
  } else {
    r.a = *reinterpret_cast<const uint2*>(row + pc.o1);
    r.b = *reinterpret_cast<const uint2*>(row + pc.o2);
  }
}
__device__ __forceinline__ void load_piece(const float* row, const Piece& pc, Raw<float>& r) {
  r.a = *reinterpret_cast<const float4*>(row + pc.o1);
  r.b = *reinterpret_cast<const float4*>(row + pc.o2);
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
  const uint2 a = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3])), b = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
  if (pc.together) {
    *reinterpret_cast<uint4*>(row + pc.o1) = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<uint2*>(row + pc.o1) = a;
    *reinterpret_cast<uint2*>(row + pc.o2) = b;
  }
}
__device__ __forceinline__ void store_piece(float* row, const Piece& pc, const float* x) {
  *reinterpret_cast<float4*>(row + pc.o1) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(row + pc.o2) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store_codes(uint8_t* row, const Piece& pc, uint32_t a, uint32_t b) {
  if (pc.together) {
    *reinterpret_cast<uint2*>(row + pc.o1) = make_uint2(a, b);
  } else {
    *reinterpret_cast<uint32_t*>(row + pc.o1) = a;
    *reinterpret_cast<uint32_t*>(row + pc.o2) = b;
  }
}
// Four codes times f1 f2.
__device__ __forceinline__ uint32_t move_codes(uint32_t w, float f1, float f2) {
  const float2 a = from_e4m3_pair(w & 0xFFFFu), b = from_e4m3_pair(w >> 16);
  return e4m3_pair(a.x * f1 * f2, a.y * f1 * f2) | e4m3_pair(b.x * f1 * f2, b.y * f1 * f2) << 16;
}

template <class T, bool Q8>
__global__ void __launch_bounds__(8 * AP_T, 2) append_kernel(const AppendP p) {
  __shared__ uint32_t s_max[Q8 ? AP_MAX : 1];              // bits of the heads' largest finite |x|
  __shared__ uint8_t s_was[Q8 ? AP_MAX : 1];               // scale bytes of the block before the call
  __shared__ int s_odd;                                    // something is not finite
  const int tid = threadIdx.x, lane = tid & 31, tokens = blockDim.x >> 3;      // tokens at a time
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
  const int item0 = blockIdx.y * p.per, item1 = min(item0 + p.per, p.items);
  Piece pc;
  {
    const int a = tid & 7;
    pc.turns = 8 * a < 2 * pairs;
    pc.together = !(halves && pc.turns);
    pc.o1 = pc.together ? 8 * a : 4 * a;
    pc.o2 = pc.together ? 8 * a + 4 : pairs + 4 * a;
  }
  const bool whole = !Q8 || p.tile <= tokens;
  const bool begins = !Q8 || t0 >= begin;                  // the block, with this call
  // 8 bits: a block lies in one page
  const int bp = Q8 ? paged_page(p.c, p.c.page_table, p.c.table_stride, slot, (int)t0) : -1;
  auto scale_at = [&](int item) {                          // of a head of keys or values
    const int h = item - nq < nk ? item - nq : item - nq - nk;
    return (item - nq < nk ? p.c.k_scale : p.c.v_scale) + scale_off(p.c, bp, h, (int)t0);
  };
  if (Q8) {
    for (int x = tid; x < item1 - item0; x += blockDim.x) {
      s_max[x] = 0u;
      s_was[x] = begins || bp < 0 || item0 + x < nq ? 0 : *scale_at(item0 + x);
    }
    if (tid == 0) s_odd = 0;
    __syncthreads();
  }
  for (int pass = whole ? 1 : 0; pass < 2; ++pass) {
    if (Q8 && !whole && pass == 1) __syncthreads();        // all largest values are known
    for (long long sub = pass == 0 ? (lo - t0) / tokens * tokens : 0; sub < p.tile && t0 + sub < hi; sub += tokens) {
      const long long t = t0 + sub + (tid >> 3);           // this thread's token
      const bool live = t >= lo && t < hi, older = Q8 && t < begin;
      const size_t row = live ? (size_t)(row0 + (t - start)) : 0;
      const int page = Q8 ? bp : live ? paged_page(p.c, p.c.page_table, p.c.table_stride, slot, (int)t) : -1;
      float cs[4], sn[4];
      bool angles = false;                                 // known
      // Heads h .. h1 - 1 of queries (0), keys (1) or values (2), of which m0 is the first one's place in s_max.
      auto heads = [&](auto kind, int h, int h1, int m0) {
        constexpr int KIND = decltype(kind)::value;
        if (h >= h1 || (KIND == 0 && pass == 0)) return;
        const T* src = (const T*)(KIND == 0 ? p.a.q : KIND == 1 ? p.a.k : p.a.v) +
                       row * (size_t)(KIND == 0 ? p.a.q_stride : KIND == 1 ? p.a.k_stride : p.a.v_stride) + (size_t)h * WS_DH;
        Raw<T> raw[AP_H];
        auto load = [&](int n) {
#pragma unroll
          for (int u = 0; u < AP_H; ++u) {
            raw[u] = Raw<T>{};
            if (u < n && live) load_piece(src + u * WS_DH, pc, raw[u]);
          }
          src += AP_H * WS_DH;
        };
        load(h1 - h);                                      // under the angles
        if (KIND < 2 && !angles && pc.turns && live) {
          const int m = p.a.pos ? p.a.pos[row] : (int)t;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t phase = (uint64_t)(int64_t)m * p.a.turns[4 * (tid & 7) + e];
            sincospif((float)(int32_t)(uint32_t)(phase >> 32) * (1.f / 2147483648.f), &sn[e], &cs[e]);
          }
        }
        if (KIND < 2) angles = true;
        T* to = KIND == 0 ? (T*)p.a.q_out + row * (size_t)p.a.q_out_stride : (T*)(KIND == 1 ? p.c.k : p.c.v);
        uint8_t* to8 = (uint8_t*)(KIND == 1 ? p.c.k : p.c.v);
        if (KIND > 0 && page >= 0 && (live || older)) {
          const size_t off = paged_off(p.c, page, 0, (int)t);
          to += off;
          to8 += off;
        }
        const size_t step = KIND == 0 ? WS_DH : (size_t)p.c.head_stride;   // from a head to the next
        to += (size_t)h * step;
        to8 += (size_t)h * step;
        for (; h < h1; h += AP_H, m0 += AP_H) {
          float x[AP_H][8];
#pragma unroll
          for (int u = 0; u < AP_H; ++u) unpack(raw[u], x[u]);
          if (h + AP_H < h1) load(h1 - h - AP_H);
          if (KIND < 2 && pc.turns) {
#pragma unroll
            for (int u = 0; u < AP_H; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // (x[2 e], x[2 e + 1]) or (x[e], x[4 + e]): the places are the compiler's to know
                const float a = halves ? x[u][e] : x[u][2 * e], b = halves ? x[u][4 + e] : x[u][2 * e + 1];
                const float v = a * cs[e] - b * sn[e], w = a * sn[e] + b * cs[e];
                if (halves) { x[u][e] = v; x[u][4 + e] = w; } else { x[u][2 * e] = v; x[u][2 * e + 1] = w; }
              }
          }
          if (KIND == 0 || !Q8) {
#pragma unroll
            for (int u = 0; u < AP_H; ++u)
              if (h + u < h1 && live && (KIND == 0 || page >= 0)) store_piece(to + u * step, pc, x[u]);
            to += AP_H * step;
            continue;
          }
          if (whole || pass == 0) {
#pragma unroll
            for (int u = 0; u < AP_H; ++u) {               // rows and heads that are not there are zero
              uint32_t m = 0u;
#pragma unroll
              for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[u][e]) & 0x7FFFFFFFu);
              m = __reduce_max_sync(0xffffffffu, live ? m : 0u);
              if (m >= 0x7F800000u) {
                s_odd = 1;
                m = 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint32_t y = __float_as_uint(x[u][e]) & 0x7FFFFFFFu;
                  if (live && y < 0x7F800000u) m = max(m, y);
                }
                m = __reduce_max_sync(0xffffffffu, m);
              }
              if (lane == 0 && h + u < h1) atomicMax(&s_max[m0 + u], m);
            }
            if (pass == 0) continue;
            __syncthreads();
          }
          const bool odd = s_odd != 0;
          if (page >= 0 && (live || older)) {
#pragma unroll
            for (int u = 0; u < AP_H; ++u) {
              if (h + u >= h1) continue;
              const int e_was = (int)s_was[m0 + u] - 127;
              const int e_now = max(e_was, scale_exponent(__uint_as_float(s_max[m0 + u])));
              uint8_t* at = to8 + u * step;
              if (live) {
                const float f = pow2(-e_now);               // 2^-127 for byte 254 is below the normal numbers
                if (odd)
#pragma unroll
                  for (int e = 0; e < 8; ++e) x[u][e] = fabsf(x[u][e]) < INFINITY ? x[u][e] : NAN;
                store_codes(at, pc, e4m3_pair(x[u][0] * f, x[u][1] * f) | e4m3_pair(x[u][2] * f, x[u][3] * f) << 16,
                            e4m3_pair(x[u][4] * f, x[u][5] * f) | e4m3_pair(x[u][6] * f, x[u][7] * f) << 16);
              } else if (e_now > e_was) {                  // earlier tokens of the block: to the new scale
                const int down = e_was - e_now, half = down / 2;
                const float f1 = pow2(half), f2 = pow2(down - half);
                const uint32_t a = *reinterpret_cast<const uint32_t*>(at + pc.o1), b = *reinterpret_cast<const uint32_t*>(at + pc.o2);
                store_codes(at, pc, move_codes(a, f1, f2), move_codes(b, f1, f2));
              }
            }
          }
          to8 += AP_H * step;
        }
      };
      heads(std::integral_constant<int, 0>(), item0, min(item1, nq), 0);
      heads(std::integral_constant<int, 1>(), max(item0 - nq, 0), min(item1 - nq, nk), max(nq - item0, 0));
      heads(std::integral_constant<int, 2>(), max(item0 - nq - nk, 0), item1 - nq - nk, max(nq + nk - item0, 0));
    }
  }
  if (!Q8 || bp < 0) return;
  for (int x = tid; x < item1 - item0; x += blockDim.x) {  // the scales: their old ones have been read
    const int e_was = (int)s_was[x] - 127, e_now = max(e_was, scale_exponent(__uint_as_float(s_max[x])));
    if (item0 + x >= nq && (begins || e_now > e_was)) *scale_at(item0 + x) = (uint8_t)(e_now + 127);
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

template <class T, bool Q8>
cudaError_t launch(const AppendP& p, dim3 grid, int tokens, cudaStream_t s) {
  append_kernel<T, Q8><<<grid, 8 * tokens, 0, s>>>(p);
  ws_count_launches(1);
  return cudaGetLastError();
}

}  // namespace

extern "C" int ws_cache_append(const ws_paged_cache* cache, const ws_append_args* args, ws_stream stream) {
  if (const char* e = check_append(cache, args)) return paged_fail(WS_EINVAL, e);
  if (args->n_req == 0 || args->total_q == 0 || args->max_q == 0) return WS_OK;
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  AppendP p = {};
  p.c = paged_copy(*cache);
  p.a = *args;
  const bool q8 = cache->dtype == WS_E4M3;
  p.items = (args->q ? args->n_heads : 0) + 2 * cache->n_kv_heads;
  // tokens at a time: 8, 16, 32 or 64 that hold the block, or some of the chunk
  int tokens = 8;
  const int want = q8 ? cache->scale_block : min(args->max_q, 32);
  while (tokens < want && tokens < AP_T) tokens *= 2;
  p.tile = q8 ? cache->scale_block : tokens;
  const long long tiles = q8 ? ((long long)args->max_q + p.tile - 2) / p.tile + 1 : (args->max_q + p.tile - 1) / p.tile;
  // Heads split over CTAs until there are 2048 threads per SM, two rounds at
  // 61-64 registers: more CTAs hide each other's chains of lengths, pages and
  // rows, and compute more angles (the same inputs again and again, in 8 bits
  // chunks of up to 2048 rows 22.8 us, half as many CTAs 25.6, twice 25.5;
  // 480 single tokens 25.4 / 24.1 / 29.5)
  const long long units = tiles * args->n_req;
  const int most = (p.items + AP_H - 1) / AP_H, least = (p.items + AP_MAX - 1) / AP_MAX;
  const long long wanted = (16ll * SMS * 16 / tokens + units - 1) / units;
  int groups = (int)max((long long)least, min((long long)most, wanted));
  p.per = ((p.items + groups - 1) / groups + AP_H - 1) / AP_H * AP_H;
  groups = (p.items + p.per - 1) / p.per;
  if (tiles > 2147483647ll || groups > 65535) return paged_fail(WS_EINVAL, "too many tiles or heads");
  const dim3 grid((unsigned)tiles, (unsigned)groups, (unsigned)args->n_req);
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = q8 ? launch<bf16, true>(p, grid, tokens, s)
                           : cache->dtype == WS_BF16 ? launch<bf16, false>(p, grid, tokens, s) : launch<float, false>(p, grid, tokens, s);
  if (e != cudaSuccess) return paged_fail(WS_ECUDA, std::string("cache append launch: ") + cudaGetErrorString(e));
  return WS_OK;
}

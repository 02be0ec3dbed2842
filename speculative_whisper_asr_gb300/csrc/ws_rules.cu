// Penalties for repeated tokens, biases and grammar masks on the logits of a
// block's rows, with the greedy choice and its log probability
// (ws_logits_rules in include/ws.h gives the formulas).
//
// One pass over the logits: every element is read once and written once (8
// bytes per element: the HBM floor).  A row belongs to one CTA, or, where
// there are few rows, to a thread-block cluster whose CTAs take contiguous
// parts of the vocabulary.
//   1. The ids that have a penalty or a bias (a few hundred of 50,000) go
//      into a hash table in shared memory, with their occurrences counted and
//      their first bias entry found by integer atomics, whose result does not
//      depend on their order; a bitmap marks them.
//   2. Their new logits are computed, one id per thread.
//   3. All other ids stream through registers, the next 16 per thread in
//      flight while 16 are masked, stored, compared and summed.  No barrier
//      stands in that loop (with the listed ids handled inside it, pass by
//      pass, barriers took half of its time).
//   4. The listed ids' logits are stored over the stream's.
// The CTAs' (largest value, lowest id, sum of exponentials) meet in the first
// CTA's shared memory (distributed shared memory), so a call is one launch
// without scratch.
//
// 864 rows of 51,866 (260 MB with masks; 64 tokens and 64 biases per row): 58
// us, 4.5 TB/s: a CTA's steps 1, 2 and 4 (about 4 us of latency) lie under
// the other CTA of its SM, and the last of three rounds is not full.  144
// rows: 15 us; one row on eight CTAs: 8 us, a chain of latencies.
#include <string>

#include "ws_internal.cuh"

namespace {

constexpr int NT = 512;                    // threads per CTA, two CTAs per SM
constexpr int Q = 4;                       // groups of 4 ids per thread and step
constexpr int MAX_CL = 8;                  // portable cluster size
constexpr uint32_t FREE = 0xFFFFFFFFu;     // hash table: no id here

// Shared memory: table (ids, counts / new logits, first bias entries), then
// the row's grammar mask and the bitmap of the listed ids, a word per 32 ids
// counted from the row's 16-byte boundary.
struct Table { int slots, words; };
inline size_t rules_smem(const Table& t) { return (size_t)t.slots * 12 + (size_t)t.words * 8; }

struct RulesStat {
  unsigned long long key;                  // argmax_key of the largest value
  float sum;                               // sum exp(y - largest)
};

__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_of(float x) { return ex2(x * LOG2E); }
// exp(y - m), with y = m giving 1 also at infinities
__device__ __forceinline__ float exp_to(float y, float m) { return y == m ? 1.0f : exp_of(y - m); }

__device__ __forceinline__ RulesStat merge(RulesStat a, RulesStat b) {
  const float ma = key_value(a.key), mb = key_value(b.key), m = fmaxf(ma, mb);
  RulesStat r;
  r.key = a.key > b.key ? a.key : b.key;
  r.sum = a.sum * exp_to(ma, m) + b.sum * exp_to(mb, m);
  return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__global__ void __launch_bounds__(NT, 2) rules_kernel(const ws_rules_args a, const Table tb, int cl, int part) {
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ RulesStat wstat[NT / 32];
  __shared__ RulesStat cstat[MAX_CL];
  uint32_t *hid = sm, *hcount = sm + tb.slots, *hbias = hcount + tb.slots, *allow = hbias + tb.slots, *listed = allow + tb.words;
  const int row = blockIdx.x / cl;
  const int i = row / a.H, j = row - i * a.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl > 1 ? cluster_rank() : 0u;
  // everything that depends on the row alone is asked for at once
  const int live = a.block_len ? a.block_len[i] : a.H;
  const int hist_len = a.history ? a.hist_len[i] : 0, bias_len = a.bias_ids ? a.bias_len[i] : 0;
  const int state = a.masks && a.mask_row ? a.mask_row[row] : -1;
  const float theta = a.repetition ? a.repetition[i] : 1.f;
  const float alpha = a.presence ? a.presence[i] : 0.f, freq = a.frequency ? a.frequency[i] : 0.f;
  if (j >= live) {                         // the whole cluster leaves
    if (rank == 0 && tid == 0) {
      if (a.target) a.target[row] = -1;
      if (a.logprob) a.logprob[row] = 0.f;
    }
    return;
  }
  if (cl > 1) cluster_arrive();            // paired with the wait before the first remote store
  const int V = a.vocab;
  const float* z = a.logits + (size_t)row * (size_t)a.ld;
  float* o = a.out + (size_t)row * (size_t)a.ld_out;
  // ids are handled in groups of four that are 16-byte aligned in the row of
  // logits: u = v + ph, groups of u
  const int ph = (int)((reinterpret_cast<uintptr_t>(z) >> 2) & 3);
  const bool ovec = (int)((reinterpret_cast<uintptr_t>(o) >> 2) & 3) == ph;
  const int lo = (int)rank * part, hi = min(lo + part, V + ph);     // part is a multiple of 4
  // groups wholly inside the row; at most one at either end is not
  const int g0 = (lo == 0 && ph ? 4 : lo) >> 2, g1 = min((lo + part) >> 2, (V + ph) >> 2);
  const float4* zp = reinterpret_cast<const float4*>(z + 4 * (g0 + tid) - ph);
  float4 next[Q];
  auto fetch = [&](int g) {
#pragma unroll
    for (int k = 0; k < Q; ++k)
      if (g + k * NT < g1) next[k] = __ldcs(zp + k * NT);
  };
  fetch(g0 + tid);
  const int hl = min(max(hist_len, 0), a.hist_stride);
  const int len = hl + (a.block ? j : 0);                           // tokens before this row
  const int from = a.window > 0 ? max(0, len - a.window) : 0;
  const int nb = min(max(bias_len, 0), a.bias_stride);
  const int32_t* ids = a.bias_ids + (size_t)i * a.bias_stride;
  auto token = [&](int p) {                // token p of the row's sequence
    return p < hl ? a.history[(size_t)i * a.hist_stride + p] : a.block[(size_t)i * a.block_stride + (p - hl) + 1];
  };
  const int t0 = from + tid < len ? token(from + tid) : -1, e0 = tid < nb ? ids[tid] : -1;
  const bool masked = state >= 0 && state < a.n_masks;
  const uint32_t* mask = a.masks + (masked ? (size_t)state * ((V + 31) / 32) : 0);
  // this CTA's words of the two bitmaps, in u: a group's four bits are in one word
  for (int w = (lo >> 5) + tid; w < min(tb.words, (hi + 31) >> 5); w += NT) {
    const int words = (V + 31) / 32;
    const uint32_t a0 = masked && w < words ? __ldg(mask + w) : FREE, a1 = masked && ph && w > 0 ? __ldg(mask + w - 1) : FREE;
    allow[w] = __funnelshift_l(a1, a0, ph);
    listed[w] = 0u;
  }
  for (int s = tid; s < tb.slots; s += NT) { hid[s] = FREE; hcount[s] = 0u; hbias[s] = FREE; }
  __syncthreads();
  // ---- 1: the listed ids of this part
  auto here = [&](int id) { return id >= 0 && id < V && id + ph >= lo && id + ph < hi; };
  auto slot = [&](int id) {                // at most half of the slots are ever taken
    uint32_t s = ((uint32_t)id * 2654435761u) >> 7 & (uint32_t)(tb.slots - 1);
    for (;;) {
      const uint32_t old = atomicCAS(&hid[s], FREE, (uint32_t)id);
      if (old == FREE) atomicOr(&listed[(id + ph) >> 5], 1u << ((id + ph) & 31));
      if (old == FREE || old == (uint32_t)id) return s;
      s = (s + 1) & (uint32_t)(tb.slots - 1);
    }
  };
  for (int p = from + tid; p < len; p += NT) {
    const int id = p == from + tid ? t0 : token(p);
    if (here(id)) atomicAdd(&hcount[slot(id)], 1u);
  }
  for (int e = tid; e < nb; e += NT) {
    const int id = e == tid ? e0 : ids[e];
    if (here(id)) atomicMin(&hbias[slot(id)], (uint32_t)e);
  }
  __syncthreads();
  // ---- 2: their logits
  float m = -INFINITY, sum = 0.f;          // this thread's largest value, its id and its sum
  int mid = 0;
  auto add = [&](const float* y, int count, auto id_of) {
    float top = -INFINITY;
    for (int k = 0; k < count; ++k) top = fmaxf(top, y[k]);
    if (top >= m && top > -INFINITY) {
      int first = 0x7FFFFFFF;
      for (int k = count - 1; k >= 0; --k)
        if (y[k] == top) first = id_of(k);  // the lowest id that has it
      if (top > m || first < mid) mid = first;
      sum *= top > m ? exp_of(m - top) : 1.f;
      m = top;
    }
    // The difference comes first: scaled to log2 units beforehand, the
    // reference's rounding would stand in every term, the largest included
    // (4e-5 of the log probability at logits near 1000), and the largest term
    // has to be 1.
    if (fabsf(m) < 1e37f) {
      if (count == 1) {
        sum += exp_of(y[0] - m);
      } else {
        float2 s2 = make_float2(0.f, 0.f);
        for (int k = 0; k + 1 < count; k += 2) {
          float2 e = __fmul2_rn(__fadd2_rn(make_float2(y[k], y[k + 1]), make_float2(-m, -m)), make_float2(LOG2E, LOG2E));
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          s2 = __fadd2_rn(s2, e);
        }
        sum += s2.x + s2.y;
      }
    } else {                               // nothing above -inf yet (a NaN still counts), infinities, lowest values
      for (int k = 0; k < count; ++k) sum += exp_to(y[k], m);
      if (m == -INFINITY && sum == sum) sum = 0.f;
    }
  };
  for (int s = tid; s < tb.slots; s += NT) {
    if (hid[s] == FREE) continue;
    const int id = (int)hid[s];
    float x = z[id];
    if (hcount[s]) {
      x = x > 0.f ? __fdiv_rn(x, theta) : __fmul_rn(x, theta);
      x = __fsub_rn(x, __fadd_rn(__fmul_rn(freq, (float)hcount[s]), alpha));
    }
    if (hbias[s] != FREE) x = __fadd_rn(x, a.bias_vals[(size_t)i * a.bias_stride + hbias[s]]);
    if (!((allow[(id + ph) >> 5] >> ((id + ph) & 31)) & 1u)) x = -INFINITY;
    hcount[s] = __float_as_uint(x);
    add(&x, 1, [&](int) { return id; });
  }
  // up to three ids at either end of the row
  if (tid < 8) {
    const int u = tid < 4 ? lo + tid : 4 * g1 + tid - 4, v = u - ph;
    const bool edge = tid < 4 ? u < 4 * g0 : u >= 4 * g0;
    if (edge && v >= 0 && v < V && u < hi && !((listed[u >> 5] >> (u & 31)) & 1u)) {
      const float x = (allow[u >> 5] >> (u & 31)) & 1u ? z[v] : -INFINITY;
      o[v] = x;
      add(&x, 1, [&](int) { return v; });
    }
  }
  __syncthreads();                         // in place, the listed ids are read before the stream stores over them
  // ---- 3: the stream
  float* op = o + 4 * (g0 + tid) - ph;
  for (int g = g0 + tid; g < g1; g += Q * NT, op += 4 * Q * NT) {
    float y[4 * Q];
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const bool on = g + k * NT < g1;
      y[4 * k] = on ? next[k].x : -INFINITY;
      y[4 * k + 1] = on ? next[k].y : -INFINITY;
      y[4 * k + 2] = on ? next[k].z : -INFINITY;
      y[4 * k + 3] = on ? next[k].w : -INFINITY;
    }
    zp += Q * NT;
    fetch(g + Q * NT);
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      if (g + k * NT >= g1) continue;
      const int w = (g + k * NT) >> 3, sh = (4 * (g + k * NT)) & 31;
      if (masked) {
        const uint32_t bits = allow[w] >> sh;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(bits & (1u << e))) y[4 * k + e] = -INFINITY;
      }
      if (ovec) {
        __stcs(reinterpret_cast<float4*>(op) + k * NT, make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) op[4 * k * NT + e] = y[4 * k + e];
      }
      const uint32_t mine = listed[w] >> sh & 15u;
      if (mine)                            // taken care of in step 2
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (mine & (1u << e)) y[4 * k + e] = -INFINITY;
    }
    add(y, 4 * Q, [&](int k) { return 4 * (g + (k >> 2) * NT) - ph + (k & 3); });
  }
  __syncthreads();
  // ---- 4: the listed ids over the stream's
  for (int s = tid; s < tb.slots; s += NT)
    if (hid[s] != FREE) o[hid[s]] = __uint_as_float(hcount[s]);
  // ---- the row's largest value (lowest id) and the sum relative to it
  RulesStat best;
  {
    const uint32_t ord = (uint32_t)(argmax_key(m, 0) >> 32), wo = __reduce_max_sync(0xffffffffu, ord);
    const uint32_t id = __reduce_min_sync(0xffffffffu, ord == wo ? (uint32_t)mid : 0xFFFFFFFFu);
    best.key = ((unsigned long long)wo << 32) | (unsigned long long)(0xFFFFFFFFu - id);
    sum *= exp_to(m, key_value(best.key));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    best.sum = sum;
  }
  if (lane == 0) wstat[warp] = best;
  __syncthreads();
  if (warp == 0) {
    RulesStat st = wstat[lane & (NT / 32 - 1)];
    const uint32_t hi_ = (uint32_t)(st.key >> 32), wo = __reduce_max_sync(0xffffffffu, hi_);
    const uint32_t lo_ = __reduce_max_sync(0xffffffffu, hi_ == wo ? (uint32_t)st.key : 0u);
    best.key = ((unsigned long long)wo << 32) | lo_;
    float s = st.sum * exp_to(key_value(st.key), key_value(best.key));
#pragma unroll
    for (int x = NT / 64; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    best.sum = s;
  }
  if (cl > 1) {
    cluster_wait();                        // every CTA of the cluster runs
    if (tid == 0) {
      uint32_t remote;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(remote) : "r"((uint32_t)__cvta_generic_to_shared(&cstat[rank])), "r"(0u));
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(best.key) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote + 8u), "f"(best.sum) : "memory");
    }
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && tid == 0) {
      best = cstat[0];
      for (int c = 1; c < cl; ++c) best = merge(best, cstat[c]);
    }
  }
  if (rank == 0 && tid == 0) {
    const bool none = key_value(best.key) == -INFINITY;
    if (a.target) a.target[row] = none ? -1 : argmax_key_id(best.key);
    if (a.logprob) a.logprob[row] = none ? -INFINITY : -logf(best.sum);
  }
}

int fail(int code, const char* msg) {
  ws_set_thread_error(msg);
  return code;
}

}  // namespace

extern "C" int ws_logits_rules(const ws_rules_args* p, ws_stream stream) {
  if (!p) return fail(WS_EINVAL, "null arguments");
  const ws_rules_args& a = *p;
  if (a.n < 0 || a.H < 0 || a.H > 16384) return fail(WS_EINVAL, "n must be >= 0 and H 0..16384");
  if (a.vocab < 1 || a.vocab > (1 << 18)) return fail(WS_EINVAL, "vocab must be 1..262144");
  if (a.n == 0 || a.H == 0) return WS_OK;
  if (!a.logits || !a.out) return fail(WS_EINVAL, "null logits or out");
  if ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.out)) & 3)
    return fail(WS_EINVAL, "logits and out must be 4-byte aligned");
  if (a.ld < a.vocab || a.ld_out < a.vocab) return fail(WS_EINVAL, "ld and ld_out must be >= vocab");
  if (a.logits == a.out && a.ld != a.ld_out) return fail(WS_EINVAL, "in place, ld_out must equal ld");
  if (a.hist_stride < 0 || a.bias_stride < 0) return fail(WS_EINVAL, "hist_stride and bias_stride must be >= 0");
  if (a.history && !a.hist_len) return fail(WS_EINVAL, "history without hist_len");
  if (a.block && a.block_stride < a.H) return fail(WS_EINVAL, "block_stride must be >= H");
  if (a.window < 0) return fail(WS_EINVAL, "window must be >= 0");
  if (a.bias_ids && (!a.bias_vals || !a.bias_len)) return fail(WS_EINVAL, "bias_ids without bias_vals or bias_len");
  if (a.masks && a.n_masks < 1) return fail(WS_EINVAL, "masks need n_masks >= 1");
  if (a.masks && !a.mask_row) return fail(WS_EINVAL, "masks without mask_row");
  if ((long long)a.n * a.H > 2147483647ll / MAX_CL) return fail(WS_EINVAL, "too many rows");
  // listed ids of a row at most: the tokens that count and the biases
  long long tokens = a.history ? a.hist_stride : 0;
  if (a.block) tokens += a.H - 1;
  if (a.window > 0) tokens = min(tokens, (long long)a.window);
  const long long most = tokens + (a.bias_ids ? a.bias_stride : 0);
  if (most > 4096) return fail(WS_EUNSUPPORTED, "more than 4096 tokens and biases per row (window limits the tokens)");
  if (a.logits != a.out && rows_overlap(a.logits, a.ld * 4, a.out, a.ld_out * 4, (long long)a.n * a.H, (int64_t)a.vocab * 4))
    return fail(WS_EINVAL, "out must be logits or share no elements with them");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return fail(WS_ECUDA, (std::string("a CUDA error was pending before this call: ") +
                           cudaGetErrorString(prior)).c_str());
  Table tb;
  tb.slots = 64;
  while (tb.slots < 2 * most) tb.slots *= 2;
  tb.words = (a.vocab + 3 + 31) / 32;
  const size_t smem = rules_smem(tb);
  // one CTA per row where that gives every SM its two; else the row is shared
  // (one row with its launch 26 us on one CTA, 20 on eight; 16 rows 25 and 22)
  const long long rows = (long long)a.n * a.H;
  const int steps = (a.vocab + 3 + 4 * Q * NT - 1) / (4 * Q * NT);
  const int cl = (int)max(1ll, min((long long)min(MAX_CL, steps), 304 / rows));
  const int part = ((a.vocab + 3 + cl - 1) / cl + 3) / 4 * 4;
  cudaError_t e = cudaFuncSetAttribute(rules_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 192 * 1024);
  if (e != cudaSuccess) return fail(WS_ECUDA, (std::string("logits rules: ") + cudaGetErrorString(e)).c_str());
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(a.n * a.H * cl));
  c.blockDim = dim3(NT);
  c.dynamicSmemBytes = smem;
  c.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cl; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, rules_kernel, a, tb, cl, part);
  if (e != cudaSuccess) return fail(WS_ECUDA, (std::string("logits rules launch: ") + cudaGetErrorString(e)).c_str());
  ws_count_launches(1);
  return WS_OK;
}

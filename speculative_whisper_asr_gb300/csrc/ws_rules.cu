// Penalties for repeated tokens, biases and grammar masks on the logits of a
// block's rows, with the greedy choice and its log probability
// (ws_logits_rules in include/ws.h gives the formulas).
//
// One pass over the logits: every element is read once and written once (8
// bytes per element: the HBM floor).  A row belongs to one CTA, or, where
// there are few rows, to a thread-block cluster whose CTAs take contiguous
// parts of the vocabulary.  Passes of 8,192 ids arrive in shared memory by
// bulk copies, the next one under the current one's work.  Beside them a
// table of the pass's ids is built,
//   word[v] = first bias entry that lists v (high half) | occurrences of v
//             in the row's token sequence (low half),
// by integer atomics, whose result does not depend on their order.  The
// penalties and biases are applied to the few listed ids alone, each claimed
// by one thread, and the dense loop only masks, stores, compares and sums
// exponentials: with the penalties inside it, unrolled over registers, the
// code was fetched from memory once per launch and cost more than the data.
// The CTAs' (largest value, lowest id, sum of exponentials) meet in the first
// CTA's shared memory (distributed shared memory), so a call is one launch
// without scratch.
#include <string>

#include "ws_tc.cuh"

namespace {

constexpr int NT = 512;                    // threads per CTA
constexpr int SPAN = 8192;                 // ids per pass
constexpr int SMEM = 3 * SPAN * 4;         // two passes of logits and the table: two CTAs per SM
constexpr int MAX_CL = 8;                  // portable cluster size
constexpr int WORDS = SPAN / 32 + 1;       // grammar mask words of a pass

struct RulesStat {
  unsigned long long key;                  // argmax_key of the largest value
  float sum;                               // sum exp(y - largest)
};

__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
// exp(y - m), with y = m giving 1 also at infinities
__device__ __forceinline__ float exp_to(float y, float m) { return y == m ? 1.0f : __expf(y - m); }

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

__global__ void __launch_bounds__(NT, 2) rules_kernel(const ws_rules_args a, int cl, int part) {
  extern __shared__ __align__(128) float ysm[];      // [2][SPAN] logits, then the table
  __shared__ uint32_t words[2][WORDS];
  __shared__ RulesStat wstat[NT / 32];
  __shared__ RulesStat cstat[MAX_CL];
  __shared__ __align__(8) uint64_t bar[2];
  uint32_t* tab = reinterpret_cast<uint32_t*>(ysm + 2 * SPAN);
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
  // whole groups inside the row come by the bulk copy, up to three ids at
  // either end of the row one by one
  auto first_whole = [&](int base) { return base == 0 && ph ? 4 : base; };
  auto end_whole = [&](int base) { return max(first_whole(base), min(base + SPAN, hi) & ~3); };
  auto copy = [&](int base, int buf) {
    const int b0 = first_whole(base), b1 = end_whole(base);
    tc::mbar_expect_tx(&bar[buf], (uint32_t)(b1 - b0) * 4u);
    if (b1 > b0) tc::bulk_g2s(ysm + buf * SPAN + (b0 - base), z + (b0 - ph), (uint32_t)(b1 - b0) * 4u, &bar[buf]);
  };
  if (tid == 0) {
    tc::mbar_init(&bar[0], 1);
    tc::mbar_init(&bar[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lo < hi) copy(lo, 0);
  }
  const uint32_t* mask = state >= 0 && state < a.n_masks ? a.masks + (size_t)state * ((V + 31) / 32) : nullptr;
  auto mask_word = [&](int base) -> uint32_t {     // this thread's word of the pass
    const int w = (max(base - ph, 0) >> 5) + tid;
    return mask && tid < WORDS && base < hi && w < (V + 31) / 32 ? __ldg(mask + w) : 0u;
  };
  const int hl = min(max(hist_len, 0), a.hist_stride);
  const int len = hl + (a.block ? j : 0);                           // tokens before this row
  const int from = a.window > 0 ? max(0, len - a.window) : 0;
  const int nb = min(max(bias_len, 0), a.bias_stride);
  const int32_t* ids = a.bias_ids + (size_t)i * a.bias_stride;
  auto token = [&](int p) {                // token p of the row's sequence
    return p < hl ? a.history[(size_t)i * a.hist_stride + p] : a.block[(size_t)i * a.block_stride + (p - hl) + 1];
  };
  // this thread's first token and bias stay in registers for every pass
  const int p0 = from + tid;
  const int t0 = p0 < len ? token(p0) : -1, e0 = tid < nb ? ids[tid] : -1;
  const float v0 = tid < nb ? a.bias_vals[(size_t)i * a.bias_stride + tid] : 0.f;
  uint32_t word = mask_word(lo);
  for (int x = tid; x < SPAN / 4; x += NT) reinterpret_cast<uint4*>(tab)[x] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  float m = -INFINITY, sum = 0.f;          // this thread's largest value, its id and its sum
  int mid = 0;
  bool dead = false;
  for (int base = lo, pass = 0; base < hi; base += SPAN, ++pass) {
    const int buf = pass & 1, n = min(base + SPAN, hi) - base;
    float* ys = ysm + buf * SPAN;
    if (base + SPAN < hi && tid == 0) copy(base + SPAN, buf ^ 1);
    if (tid < WORDS) words[buf][tid] = word;
    word = mask_word(base + SPAN);
    if (tid < 8) {
      const int b0 = first_whole(base), b1 = end_whole(base);
      const int u = tid < 4 ? base + tid : b1 + tid - 4, v = u - ph;
      if (u >= base && u < base + SPAN && (u < b0 || u >= b1)) ys[u - base] = v >= 0 && v < V && u < base + n ? z[v] : -INFINITY;
    }
    const int shift = ph - base;
    auto here = [&](int id) { return id >= 0 && id < V && id + shift >= 0 && id + shift < n; };
    if (nb > 0) {
      for (int e = tid; e < nb; e += NT) {
        const int id = e == tid ? e0 : ids[e];
        if (here(id)) atomicMax(&tab[id + shift], (uint32_t)(0xFFFF - e) << 16);
      }
      __syncthreads();
    }
    for (int p = p0; p < len; p += NT) {
      const int id = p == p0 ? t0 : token(p);
      if (here(id)) atomicAdd(&tab[id + shift], 1u);
    }
    __syncthreads();
    if (!tc::mbar_wait(&bar[buf], (uint32_t)((pass >> 1) & 1))) {   // ran out: say so, and see the copy land
      dead = true;
      tc::mbar_wait(&bar[buf], (uint32_t)((pass >> 1) & 1));
    }
    // ---- penalties: the thread that takes an id's count away applies it
    for (int p = p0; p < len; p += NT) {
      const int id = p == p0 ? t0 : token(p);
      if (!here(id)) continue;
      const uint32_t c = atomicAnd(&tab[id + shift], 0xFFFF0000u) & 0xFFFFu;
      if (c) {
        float x = ys[id + shift];
        x = x > 0.f ? __fdiv_rn(x, theta) : __fmul_rn(x, theta);
        ys[id + shift] = __fsub_rn(x, __fadd_rn(__fmul_rn(freq, (float)c), alpha));
      }
    }
    __syncthreads();
    if (nb > 0) {
      for (int e = tid; e < nb; e += NT) {
        const int id = e == tid ? e0 : ids[e];
        if (here(id) && tab[id + shift] >> 16 == (uint32_t)(0xFFFF - e)) {
          ys[id + shift] = __fadd_rn(ys[id + shift], e == tid ? v0 : a.bias_vals[(size_t)i * a.bias_stride + e]);
          tab[id + shift] = 0u;            // the entry that won leaves the word clear for the next pass
        }
      }
      __syncthreads();
    }
    // ---- mask, store, compare, sum
    const int w0 = max(base - ph, 0) >> 5;
#pragma unroll 2
    for (int x = tid; x < (n + 3) / 4; x += NT) {
      float4 y = reinterpret_cast<const float4*>(ys)[x];
      const int v = base + 4 * x - ph;
      const bool whole = v >= 0 && v + 3 < V;
      if (mask) {
        // bits of ids below 0 or at V and above are of no consequence: those logits are -inf already
        const int s = max(v, 0), w = (s >> 5) - w0;
        const uint32_t bits = __funnelshift_r(words[buf][w], words[buf][min(w + 1, WORDS - 1)], s & 31) << (s - v);
        y.x = bits & 1u ? y.x : -INFINITY;
        y.y = bits & 2u ? y.y : -INFINITY;
        y.z = bits & 4u ? y.z : -INFINITY;
        y.w = bits & 8u ? y.w : -INFINITY;
      }
      if (whole && ovec) {
        __stcs(reinterpret_cast<float4*>(o + v), y);
      } else {
        if (v >= 0 && v < V) o[v] = y.x;
        if (v + 1 >= 0 && v + 1 < V) o[v + 1] = y.y;
        if (v + 2 >= 0 && v + 2 < V) o[v + 2] = y.z;
        if (v + 3 >= 0 && v + 3 < V) o[v + 3] = y.w;
      }
      const float top = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
      if (top > m) {
        sum *= __expf(m - top);
        m = top;
        mid = y.x == top ? v : y.y == top ? v + 1 : y.z == top ? v + 2 : v + 3;
      }
      if (fabsf(m) < INFINITY) {
        sum += (__expf(y.x - m) + __expf(y.y - m)) + (__expf(y.z - m) + __expf(y.w - m));
      } else {                             // nothing above -inf yet (a NaN still counts), or a row with +inf
        sum += (exp_to(y.x, m) + exp_to(y.y, m)) + (exp_to(y.z, m) + exp_to(y.w, m));
        if (m < 0.f && sum == sum) sum = 0.f;
      }
    }
    if (base + SPAN < hi) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before a later copy over these logits
      __syncthreads();
    }
  }
  // ---- the row's largest value (lowest id) and the sum relative to it
  RulesStat best;
  {
    const uint32_t ord = (uint32_t)(argmax_key(m, 0) >> 32), wo = __reduce_max_sync(0xffffffffu, ord);
    const uint32_t id = __reduce_min_sync(0xffffffffu, ord == wo ? (uint32_t)mid : 0xFFFFFFFFu);
    best.key = ((unsigned long long)wo << 32) | (unsigned long long)(0xFFFFFFFFu - id);
    sum *= exp_to(m, key_value(best.key));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    best.sum = __any_sync(0xffffffffu, dead) ? NAN : sum;
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
  if (a.vocab < 1 || a.vocab > (1 << 24)) return fail(WS_EINVAL, "vocab must be 1..2^24");
  if (a.n == 0 || a.H == 0) return WS_OK;
  if (!a.logits || !a.out) return fail(WS_EINVAL, "null logits or out");
  if ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.out)) & 3)
    return fail(WS_EINVAL, "logits and out must be 4-byte aligned");
  if (a.ld < a.vocab || a.ld_out < a.vocab) return fail(WS_EINVAL, "ld and ld_out must be >= vocab");
  if (a.logits == a.out && a.ld != a.ld_out) return fail(WS_EINVAL, "in place, ld_out must equal ld");
  if (a.hist_stride < 0 || a.hist_stride > 32768) return fail(WS_EINVAL, "hist_stride must be 0..32768");
  if (a.history && !a.hist_len) return fail(WS_EINVAL, "history without hist_len");
  if (a.block && a.block_stride < a.H) return fail(WS_EINVAL, "block_stride must be >= H");
  if (a.window < 0) return fail(WS_EINVAL, "window must be >= 0");
  if (a.bias_stride < 0 || a.bias_stride > 32768) return fail(WS_EINVAL, "bias_stride must be 0..32768");
  if (a.bias_ids && (!a.bias_vals || !a.bias_len)) return fail(WS_EINVAL, "bias_ids without bias_vals or bias_len");
  if (a.masks && a.n_masks < 1) return fail(WS_EINVAL, "masks need n_masks >= 1");
  if (a.masks && !a.mask_row) return fail(WS_EINVAL, "masks without mask_row");
  if ((long long)a.n * a.H > 2147483647ll / MAX_CL) return fail(WS_EINVAL, "too many rows");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return fail(WS_ECUDA, (std::string("a CUDA error was pending before this call: ") +
                           cudaGetErrorString(prior)).c_str());
  // one CTA per row where that gives every SM its two; else the row is shared
  const long long rows = (long long)a.n * a.H;
  const int passes = (a.vocab + 3 + SPAN - 1) / SPAN;
  const int cl = (int)max(1ll, min((long long)min(MAX_CL, passes), 304 / rows));
  const int part = ((a.vocab + 3 + cl - 1) / cl + 3) / 4 * 4;
  cudaError_t e = cudaFuncSetAttribute(rules_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return fail(WS_ECUDA, (std::string("logits rules: ") + cudaGetErrorString(e)).c_str());
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(a.n * a.H * cl));
  c.blockDim = dim3(NT);
  c.dynamicSmemBytes = SMEM;
  c.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cl; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, rules_kernel, a, cl, part);
  if (e != cudaSuccess) return fail(WS_ECUDA, (std::string("logits rules launch: ") + cudaGetErrorString(e)).c_str());
  ws_count_launches(1);
  return WS_OK;
}

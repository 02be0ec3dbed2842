// Penalties for repeated tokens, biases and grammar masks on the logits of a
// block's rows, with the greedy choice and its log probability
// (ws_logits_rules in include/ws.h gives the formulas).
//
// One pass over the logits: every element is read once, changed in
// registers and written once (8 bytes per element: the HBM floor).  A row
// belongs to one thread-block cluster whose CTAs take contiguous parts of
// the vocabulary; each CTA issues all its logit loads first, then builds a
// table of its part in shared memory while they are in flight,
//   word[v] = first bias entry that lists v (high half) | occurrences of v
//             in the row's token sequence (low half),
// by integer atomics, whose result does not depend on their order.  Almost
// every word is 0, so an element costs one shared load and a test.  The
// CTAs' (largest value, lowest id, sum of exponentials) meet in the first
// CTA's shared memory (distributed shared memory), so a call is one launch
// without scratch.
#include <string>

#include "ws_internal.cuh"

namespace {

constexpr int NT = 256;                    // threads per CTA
constexpr int GPT = 8;                     // groups of 4 logits per thread and pass
constexpr int SPAN = NT * GPT * 4;         // ids per pass of a CTA (a 32 KB table)
constexpr int MAX_CL = 8;                  // portable cluster size

struct RulesStat {
  unsigned long long key;                  // argmax_key of the largest value
  float sum;                               // sum exp(y - largest)
};

__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
// exp(y - m) with y = m giving 1 also at infinities
__device__ __forceinline__ float exp_to(float y, float m) { return y == m ? 1.0f : __expf(y - m); }

__device__ __forceinline__ RulesStat merge(RulesStat a, RulesStat b) {
  const float ma = key_value(a.key), mb = key_value(b.key), m = fmaxf(ma, mb);
  RulesStat r;
  r.key = a.key > b.key ? a.key : b.key;
  r.sum = a.sum * (a.sum > 0.f ? exp_to(ma, m) : 0.f) + b.sum * (b.sum > 0.f ? exp_to(mb, m) : 0.f);
  return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__global__ void __launch_bounds__(NT) rules_kernel(const ws_rules_args a, int cl, int part) {
  __shared__ __align__(16) uint32_t tab[SPAN];
  __shared__ RulesStat wstat[NT / 32];
  __shared__ RulesStat cstat[MAX_CL];
  const int row = blockIdx.x / cl;
  const int i = row / a.H, j = row - i * a.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl > 1 ? cluster_rank() : 0u;
  const int live = a.block_len ? a.block_len[i] : a.H;
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
  const int u_end = V + ph;
  const int lo = (int)rank * part, hi = min(lo + part, u_end);      // part is a multiple of 4
  const float theta = a.repetition ? a.repetition[i] : 1.f;
  const float alpha = a.presence ? a.presence[i] : 0.f, freq = a.frequency ? a.frequency[i] : 0.f;
  const float* bvals = a.bias_vals ? a.bias_vals + (size_t)i * a.bias_stride : nullptr;
  const uint32_t* mask = nullptr;
  if (a.masks && a.mask_row) {
    const int s = a.mask_row[row];
    if (s >= 0 && s < a.n_masks) mask = a.masks + (size_t)s * ((V + 31) / 32);
  }
  const int hl = a.history ? min(max(a.hist_len[i], 0), a.hist_stride) : 0;
  const int len = hl + (a.block ? j : 0);                           // tokens before this row
  const int from = a.window > 0 ? max(0, len - a.window) : 0;
  const int nb = a.bias_ids ? min(max(a.bias_len[i], 0), a.bias_stride) : 0;

  RulesStat best;
  best.key = argmax_key(-INFINITY, 0);
  best.sum = 0.f;
  for (int base = lo; base < hi; base += SPAN) {
    float y[GPT][4];
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      const int u = base + (g * NT + tid) * 4, v = u - ph;
      if (u < hi && v >= 0 && v + 3 < V) {
        const float4 q = __ldcs(reinterpret_cast<const float4*>(z + v));
        y[g][0] = q.x; y[g][1] = q.y; y[g][2] = q.z; y[g][3] = q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[g][e] = (u < hi && v + e >= 0 && v + e < V) ? z[v + e] : -INFINITY;
      }
    }
    // ---- the table of ids base - ph .. + SPAN - 1
#pragma unroll
    for (int g = 0; g < GPT; ++g) reinterpret_cast<uint4*>(tab)[g * NT + tid] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    const int end = min(base + SPAN, hi);
    if (nb > 0) {
      const int32_t* ids = a.bias_ids + (size_t)i * a.bias_stride;
      for (int e = tid; e < nb; e += NT) {
        const int u = ids[e] + ph;
        if (ids[e] >= 0 && ids[e] < V && u >= base && u < end) atomicMax(&tab[u - base], (uint32_t)(0xFFFF - e) << 16);
      }
      __syncthreads();
    }
    for (int p = from + tid; p < len; p += NT) {
      const int t = p < hl ? a.history[(size_t)i * a.hist_stride + p] : a.block[(size_t)i * a.block_stride + (p - hl) + 1];
      const int u = t + ph;
      if (t >= 0 && t < V && u >= base && u < end) atomicAdd(&tab[u - base], 1u);
    }
    __syncthreads();
    // ---- the new logits
    float m = -INFINITY;
    int id = 0;
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      const int u = base + (g * NT + tid) * 4, v = u - ph;
      if (u >= hi) break;
      const uint4 w4 = reinterpret_cast<const uint4*>(tab)[g * NT + tid];
      if (w4.x | w4.y | w4.z | w4.w) {
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t c = w[e] & 0xFFFFu, b = w[e] >> 16;
          float x = y[g][e];
          if (c) {
            x = x > 0.f ? __fdiv_rn(x, theta) : __fmul_rn(x, theta);
            x = __fsub_rn(x, __fadd_rn(__fmul_rn(freq, (float)c), alpha));
          }
          if (b) x = __fadd_rn(x, bvals[0xFFFFu - b]);
          y[g][e] = x;
        }
      }
      const bool whole = v >= 0 && v + 3 < V;
      if (mask) {
        uint32_t bits;
        if (whole) {
          const int sh = v & 31;
          uint32_t w0 = __ldg(mask + (v >> 5)), w1 = sh > 28 ? __ldg(mask + (v >> 5) + 1) : 0u;
          bits = __funnelshift_r(w0, w1, sh);
        } else {
          bits = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (v + e >= 0 && v + e < V) bits |= ((__ldg(mask + ((v + e) >> 5)) >> ((v + e) & 31)) & 1u) << e;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[g][e] = (bits >> e) & 1u ? y[g][e] : -INFINITY;
      }
      if (whole && ovec) {
        __stcs(reinterpret_cast<float4*>(o + v), make_float4(y[g][0], y[g][1], y[g][2], y[g][3]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v + e >= 0 && v + e < V) o[v + e] = y[g][e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (v + e < 0 || v + e >= V) { y[g][e] = -INFINITY; continue; }
        if (y[g][e] > m) { m = y[g][e]; id = v + e; }
      }
    }
    // ---- this pass's largest value and, relative to it, the sum
    unsigned long long key = argmax_key(m, id);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, s);
      key = other > key ? other : key;
    }
    const float wm = key_value(key);
    float sum = 0.f;
    if (a.logprob && wm > -INFINITY) {
#pragma unroll
      for (int g = 0; g < GPT; ++g) {
        if (base + (g * NT + tid) * 4 >= hi) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += exp_to(y[g][e], wm);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    }
    RulesStat st;
    st.key = key; st.sum = sum;
    best = merge(best, st);
    __syncthreads();                       // the table is rebuilt by the next pass
  }
  if (lane == 0) wstat[warp] = best;
  __syncthreads();
  if (warp == 0) {
    RulesStat st = wstat[lane & (NT / 32 - 1)];
#pragma unroll
    for (int s = 1; s < NT / 32; s <<= 1) {
      RulesStat other;
      other.key = __shfl_xor_sync(0xffffffffu, st.key, s);
      other.sum = __shfl_xor_sync(0xffffffffu, st.sum, s);
      st = (lane & s) ? merge(other, st) : merge(st, other);
    }
    best = st;
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
  // a CTA's loads fit one pass where the cluster limit allows it
  const int cl = min(MAX_CL, (a.vocab + 3 + SPAN - 1) / SPAN);
  const int part = ((a.vocab + 3 + cl - 1) / cl + 3) / 4 * 4;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(a.n * a.H * cl));
  c.blockDim = dim3(NT);
  c.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cl; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, rules_kernel, a, cl, part);
  if (e != cudaSuccess) return fail(WS_ECUDA, (std::string("logits rules launch: ") + cudaGetErrorString(e)).c_str());
  ws_count_launches(1);
  return WS_OK;
}

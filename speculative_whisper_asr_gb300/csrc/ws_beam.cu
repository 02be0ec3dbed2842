// One step of beam search over beams and vocabulary (ws_beam_select in
// include/ws.h gives the rule).
//
// scan_kernel.  A CTA reads a part of one beam's logits once: a running
// maximum with the sum of exponentials below it, and each thread's largest
// logit.  A thread's logits depend on the tokens alone, not on the row's
// alignment, so equal rows get equal sums and equal candidates stay equal.
// The K = beams + 1 best candidates of a part (no beam can need more: `beams`
// that go on and the end) are found after the stream, without a barrier or a
// list in it: T, the K-th best of the threads' best in the order (larger
// logit, lower token), has K logits at or before it, so each of the K best is
// in a thread whose best is not behind T, and exactly K threads are such.
// Their logits (K of the 128th parts, from L2) are read again, those not
// behind T kept, and ranked by counting.
//
// merge_kernel.  One CTA per request: log-sum-exps of the beams, candidates'
// scores as two fp32 numbers each (what differs from another beam's by less
// than fp32's step is still told apart), the parts' candidates in order within
// their beams, the beams' against each other by whole numbers that order like
// the scores, and the 2 * beams best dealt out: those that end go to the
// finished transcripts.  Then each thread moves a column of the transcripts for
// all beams, so the move may be in place.
// 96 requests x 5 beams over 51,866 tokens (100 MB): 33 us, of which the scan,
// one round of CTAs, takes 23 (4.4 TB/s) and the merge 8, a chain of latencies
// (80 registers and four bytes spilled); one request 14.
#include <string>

#include "ws_paged.cuh"

namespace {

constexpr int BM_NT = 128;                  // threads per part ...
constexpr int BM_MT = 256;                  // ... and per request
constexpr int BM_BEAMS = 16;
constexpr int BM_K = BM_BEAMS + 1;
constexpr int BM_W = BM_NT / 32;
constexpr int BM_STEP = 2 * BM_NT;         // logits of a step of all threads
constexpr int BM_PART = 32768;             // logits per part, at most
constexpr int BM_PARTS = 32;               // parts per row, at most (a lane each in the merge)
constexpr float LOG2E = 1.4426950408889634f;

struct BeamP {
  ws_beam_args a;
  int parts, part;                         // per row; logits per part
  unsigned long long* cand;                // [rows][parts][K] argmax keys, 0: none
  float2* stat;                            // [rows][parts] (largest logit, sum of exp below it)
};

// The difference comes first: log2(e) times each of the two, one of them
// rounded, would put an error of the logits' own size into every term.
__device__ __forceinline__ float exp_of(float difference) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(difference * LOG2E));
  return y;
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
// Scores are sums of two fp32 numbers, hi the sum rounded and lo what is left
// (double is 64 times slower here: 10 of the merge's 15 us were its sums).
struct Two { float hi, lo; };
__device__ __forceinline__ Two two_sum(float a, float b) {           // exact (Knuth)
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two plus(Two a, float b) {
  const Two s = two_sum(a.hi, b);
  const float lo = __fadd_rn(s.lo, a.lo), hi = __fadd_rn(s.hi, lo);
  return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}
// x - log(y), y > 0: exponent and significand (0.75 .. 1.5) of y apart, with log 2 in a part whose multiples are exact
// and the rest (Cody and Waite's reduction); good to 2^-24 of the significand's logarithm.
__device__ __forceinline__ Two less_log(Two x, float y) {
  const int e = (int)(__float_as_uint(y) - 0x3F400000u) >> 23;
  const float f = __uint_as_float(__float_as_uint(y) - ((uint32_t)e << 23));
  return plus(plus(x, -(float)e * 0.693115234375f), -fmaf((float)e, 3.1946184945e-05f, logf(f)));
}
__device__ __forceinline__ unsigned long long two_order(Two x) {     // larger score, larger number
  return (unsigned long long)f32_order(x.hi == 0.f ? 0.f : x.hi) << 32 | f32_order(x.lo == 0.f ? 0.f : x.lo);
}
__device__ __forceinline__ bool idle(const ws_beam_args& a, int i) {
  const bool full = a.n_done && a.n_done[i] >= a.max_done;
  return (a.tokens && a.length[i] >= a.capacity) || full;  // both asked for at once
}

// Tokens v and v + 1 of a row, -inf behind v1.  PAIR: every row is 8-byte aligned.
template <bool PAIR>
__device__ __forceinline__ float2 two_logits(const float* z, int v, int v1) {
  if (PAIR && v + 1 < v1) return __ldg(reinterpret_cast<const float2*>(z + v));
  return make_float2(v < v1 ? __ldg(z + v) : -INFINITY, v + 1 < v1 ? __ldg(z + v + 1) : -INFINITY);
}

// A thread's tokens are the same with and without PAIR: 2 tid, 2 tid + 1 and on by STEP.
template <bool PAIR>
__global__ void __launch_bounds__(BM_NT) scan_kernel(const BeamP p) {
  extern __shared__ unsigned long long s_list[];           // [K][a thread's logits]
  __shared__ unsigned long long s_key[BM_W * BM_K];
  __shared__ int s_thread[BM_K];
  __shared__ unsigned long long s_t;
  __shared__ int s_n;
  __shared__ float s_m[BM_W], s_s[BM_W];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.y, V = p.a.vocab, K = p.a.beams + 1;
  pdl_trigger();
  if (idle(p.a, row / p.a.beams)) return;
  const float* z = p.a.logits + (size_t)row * (size_t)p.a.ld;
  const int v0 = blockIdx.x * p.part, v1 = min(V, v0 + p.part);
  // ---- the stream: 2 U logits of a thread under way while 2 U are summed
  float m = -INFINITY, ref = 0.f, s = 0.f; // largest so far (ref: 0 until there is one); sum of exp(. - ref)
  int at = -1;                             // its token
  constexpr int U = 8;
  float2 next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) next[u] = two_logits<PAIR>(z, v0 + 2 * tid + u * BM_STEP, v1);
  for (int v = v0 + 2 * tid; v < v1; v += U * BM_STEP) {
    float2 f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) f[u] = next[u];
    if (v + U * BM_STEP < v1)
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = two_logits<PAIR>(z, v + (U + u) * BM_STEP, v1);
    float t = fmaxf(f[0].x, f[0].y);
#pragma unroll
    for (int u = 1; u < U; ++u) t = fmaxf(t, fmaxf(f[u].x, f[u].y));
    if (t > m) {
#pragma unroll
      for (int u = U - 1; u >= 0; --u) {
        if (f[u].y == t) at = v + u * BM_STEP + 1;
        if (f[u].x == t) at = v + u * BM_STEP;
      }
      s *= exp_of(m - t);                  // m = -inf: 0
      m = ref = t;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s += exp_of(f[u].x - ref) + exp_of(f[u].y - ref);
  }
  // ---- the K best of the warp's threads, then of the CTA's
  const unsigned long long key = at >= 0 ? argmax_key(m, at) : 0ull;
  uint32_t left = (uint32_t)(key >> 32);
  for (int r = 0; r < K; ++r) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, left);
    const uint32_t low = __reduce_max_sync(0xffffffffu, left == best ? (uint32_t)key : 0u);
    if (lane == 0) s_key[warp * K + r] = best ? (unsigned long long)best << 32 | low : 0ull;
    if (left == best && (uint32_t)key == low) left = 0u;
  }
  {
    const float wm = warp_max(m);
    const float ws = warp_sum(m > -INFINITY ? s * exp_of(m - wm) : s);
    if (lane == 0) { s_m[warp] = wm; s_s[warp] = ws; }
  }
  if (tid == 0) { s_n = 0; s_t = 1ull; }
  if (tid < K) s_thread[tid] = -1;
  __syncthreads();
  if (tid < BM_W * K) {
    const unsigned long long mine = s_key[tid];
    if (mine) {
      int rank = 0;
      for (int j = 0; j < BM_W * K; ++j) rank += s_key[j] > mine;
      if (rank < K) s_thread[rank] = (argmax_key_id(mine) - v0) % BM_STEP / 2;
      if (rank == K - 1) s_t = mine;       // else fewer than K threads have any: all that is above -inf
    }
  }
  if (tid == 0) {
    float M = s_m[0];
    for (int w = 1; w < BM_W; ++w) M = fmaxf(M, s_m[w]);
    float S = 0.f;
    for (int w = 0; w < BM_W; ++w) S += s_m[w] > -INFINITY ? s_s[w] * exp_of(s_m[w] - M) : s_s[w];
    p.stat[(size_t)row * p.parts + blockIdx.x] = make_float2(M, S);
  }
  __syncthreads();
  // ---- the logits of those threads, again
  const unsigned long long T = s_t;
  const int steps = (v1 - v0 + BM_STEP - 1) / BM_STEP;
  for (int y0 = tid; y0 < K * steps; y0 += 4 * BM_NT) {
    float2 f[4];
    int v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int y = y0 + q * BM_NT, r = y / steps, th = y < K * steps ? s_thread[r] : -1;
      v[q] = th < 0 ? v1 : v0 + (y - r * steps) * BM_STEP + 2 * th;
      f[q] = two_logits<PAIR>(z, v[q], v1);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (f[q].x > -INFINITY) {
        const unsigned long long mine = argmax_key(f[q].x, v[q]);
        if (mine >= T) s_list[atomicAdd(&s_n, 1)] = mine;
      }
      if (f[q].y > -INFINITY) {
        const unsigned long long mine = argmax_key(f[q].y, v[q] + 1);
        if (mine >= T) s_list[atomicAdd(&s_n, 1)] = mine;
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  unsigned long long* out = p.cand + ((size_t)row * p.parts + blockIdx.x) * K;
  for (int y = tid; y < n; y += BM_NT) {
    const unsigned long long mine = s_list[y];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += s_list[j] > mine;
    if (rank < K) out[rank] = mine;
  }
  if (tid >= n && tid < K) out[tid] = 0ull;
}

__global__ void __launch_bounds__(BM_MT) merge_kernel(const BeamP p) {
  extern __shared__ unsigned long long sm[];               // the parts' candidates [beams][parts * K]
  __shared__ unsigned long long s_c[BM_BEAMS * BM_K];      // a beam's K best: order of the score, 0: none
  __shared__ int s_v[BM_BEAMS * BM_K];                     // and their tokens, with the beam << 18
  __shared__ int s_top[2 * BM_BEAMS];                      // the best of all: places in s_c
  __shared__ int s_par[BM_BEAMS], s_tok[BM_BEAMS], s_dpar[BM_BEAMS], s_dplace[BM_BEAMS], s_ends;
  constexpr uint32_t ALL = 0xffffffffu;
  const ws_beam_args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = blockIdx.x, B = a.beams, K = B + 1, each = p.parts * K;
  const bool rest = idle(a, i);
  const int L = a.tokens ? max(a.length[i], 0) : 0, had = a.n_done ? max(a.n_done[i], 0) : 0;
  if (tid < 2 * BM_BEAMS) s_top[tid] = -1;
  if (tid < BM_BEAMS) { s_par[tid] = tid; s_tok[tid] = -1; }
  if (tid == 0) s_ends = 0;
  pdl_wait();
  float kept = 0.f;
  if (rest && tid < B) kept = a.score[(size_t)i * B + tid];
  if (!rest) {
    for (int b = warp; b < B; b += BM_MT / 32) {           // a warp per beam, a lane per part
      unsigned long long* list = sm + b * each;
      for (int x = lane; x < each; x += 32) list[x] = p.cand[((size_t)i * B + b) * each + x];
      const float was = a.score[(size_t)i * B + b];
      const float2 st = lane < p.parts ? p.stat[((size_t)i * B + b) * p.parts + lane] : make_float2(-INFINITY, 0.f);
      const float M = warp_max(st.x);
      const float S = warp_sum(st.x > -INFINITY ? st.y * exp_of(st.x - M) : st.y);
      const bool live = fabsf(was) < INFINITY && fabsf(M) < INFINITY && S < INFINITY;
      const Two off = live ? less_log(two_sum(was, -M), S) : Two{0.f, 0.f};
      __syncwarp();
      // the parts' lists are in order: their heads are compared K times
      unsigned long long head = lane < p.parts ? list[lane * K] : 0ull, mine = 0ull;
      int at = 0;
      for (int r = 0; r < K; ++r) {
        const uint32_t hi = __reduce_max_sync(ALL, (uint32_t)(head >> 32));
        const uint32_t lo = __reduce_max_sync(ALL, (uint32_t)(head >> 32) == hi ? (uint32_t)head : 0u);
        const unsigned long long best = (unsigned long long)hi << 32 | lo;
        if (lane == r) mine = best;
        if (best && head == best) { ++at; head = at < K ? list[lane * K + at] : 0ull; }
      }
      if (lane < K) {
        const Two c = plus(off, key_value(mine));
        s_c[b * K + lane] = live && mine && fabsf(c.hi) < INFINITY ? two_order(c) : 0ull;
        s_v[b * K + lane] = mine ? b << 18 | argmax_key_id(mine) : 0;
      }
    }
    __syncthreads();
    for (int x = tid; x < B * K; x += BM_MT) {
      const unsigned long long mine = s_c[x];
      if (!mine) continue;
      // equal scores: the lower beam, then the lower token (logits apart may come out equal)
      const int tie = s_v[x];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < B * K; ++j) {
        const unsigned long long o = s_c[j];
        rank += (o > mine) | ((o == mine) & (s_v[j] < tie));
      }
      if (rank < 2 * B) s_top[rank] = x;
    }
    __syncthreads();
    if (warp == 0) {                                       // lane = rank: which go on, which end
      const int x = lane < 2 * B ? s_top[lane] : -1;
      const int beam = x >= 0 ? s_v[x] >> 18 : 0, v = x >= 0 ? s_v[x] & 0x3FFFF : -1;
      const bool end = x >= 0 && v == a.eos_id;
      const uint32_t lives = __ballot_sync(ALL, x >= 0 && !end), below = (1u << lane) - 1u;
      const int before = __popc(lives & below);            // beams found before this candidate
      const uint32_t endings = __ballot_sync(ALL, end && before < B && a.n_done);
      const int place = had + __popc(endings & below);
      const float score = x >= 0 ? key_value(s_c[x]) : -INFINITY;
      if (x >= 0 && !end && before < B) {
        s_par[before] = beam;
        s_tok[before] = v;
        a.score_out[(size_t)i * B + before] = score;
      }
      if (((endings >> lane) & 1u) && place < a.max_done) {
        s_dpar[place - had] = beam;
        s_dplace[place - had] = place;
        a.done_score[(size_t)i * a.max_done + place] = score;
        if (a.done_length) a.done_length[(size_t)i * a.max_done + place] = L;
      }
      if (lane < B && lane >= __popc(lives)) a.score_out[(size_t)i * B + lane] = -INFINITY;
      if (lane == 0) s_ends = min(__popc(endings), a.n_done ? a.max_done - had : 0);
    }
  } else if (tid < B) {
    a.score_out[(size_t)i * B + tid] = kept;
  }
  __syncthreads();
  if (tid < B) {
    a.parent[(size_t)i * B + tid] = s_par[tid];
    a.token[(size_t)i * B + tid] = s_tok[tid];
  }
  const int ends = s_ends;
  if (tid == 0) {
    if (a.n_done) a.n_done_out[i] = rest ? a.n_done[i] : had + ends;
    if (a.tokens) a.length_out[i] = rest ? a.length[i] : L + 1;
  }
  if (!a.tokens || (rest && a.tokens == a.tokens_out)) return;
  // ---- transcripts, a column of all beams per thread
  const size_t cap = (size_t)a.capacity;
  const int32_t* src = a.tokens + (size_t)i * B * cap;
  int32_t* dst = a.tokens_out + (size_t)i * B * cap;
  const int cols = min(L, a.capacity);
  for (int t = tid; t < cols; t += BM_MT) {
    int32_t r[BM_BEAMS];
#pragma unroll
    for (int b = 0; b < BM_BEAMS; ++b)
      if (b < B) r[b] = src[(size_t)s_par[b] * cap + t];
    if (a.done_tokens)
      for (int d = 0; d < ends; ++d)
        a.done_tokens[((size_t)i * a.max_done + s_dplace[d]) * cap + t] = src[(size_t)s_dpar[d] * cap + t];
#pragma unroll
    for (int b = 0; b < BM_BEAMS; ++b)
      if (b < B) dst[(size_t)b * cap + t] = r[b];
  }
  if (!rest && tid < B) dst[(size_t)tid * cap + L] = s_tok[tid];
}

int fail(int code, const char* msg) {
  ws_set_thread_error(msg);
  return code;
}

bool apart(const void* a, const void* b, long long bytes_a, long long bytes_b) {
  const char *x = (const char*)a, *y = (const char*)b;
  return !x || !y || bytes_a <= 0 || bytes_b <= 0 || x + bytes_a <= y || y + bytes_b <= x;
}

const char* check_beam(const ws_beam_args* a) {
  if (!a) return "null arguments";
  if (a->n < 0) return "n must be >= 0";
  if (a->beams < 1 || a->beams > BM_BEAMS) return "beams must be 1..16";
  if (a->vocab < 1 || a->vocab > (1 << 18)) return "vocab must be 1..262144";
  if ((long long)a->n * a->beams > 65535) return "n * beams must be at most 65535";
  if (a->eos_id < -1 || a->eos_id >= a->vocab) return "eos_id must be -1..vocab - 1";
  if (a->max_done < 0) return "max_done must be >= 0";
  if (a->n == 0) return nullptr;
  if (!a->logits || !a->score || !a->score_out || !a->parent || !a->token) return "null logits, score, score_out, parent or token";
  if (reinterpret_cast<uintptr_t>(a->logits) & 3) return "logits must be 4-byte aligned";
  if (a->ld < a->vocab) return "ld must be >= vocab";
  if (a->tokens) {
    if (!a->tokens_out || !a->length || !a->length_out) return "tokens without tokens_out, length or length_out";
    if (a->capacity < 1) return "capacity must be >= 1";
  } else if (a->tokens_out || a->length || a->length_out || a->done_tokens || a->done_length) {
    return "lengths and transcripts need tokens";
  }
  if (a->n_done) {
    if (!a->n_done_out) return "n_done without n_done_out";
    if (a->max_done > 0 && !a->done_score) return "n_done without done_score";
  } else if (a->n_done_out || a->done_score || a->done_length || a->done_tokens) {
    return "finished transcripts need n_done";
  }
  const long long rows = 4ll * a->n * a->beams, reqs = 4ll * a->n, text = a->tokens ? rows * a->capacity : 0;
  auto in_place = [](const void* in, const void* out, long long bytes) { return in == out || apart(in, out, bytes, bytes); };
  if (!in_place(a->score, a->score_out, rows) || !in_place(a->tokens, a->tokens_out, text) ||
      !in_place(a->length, a->length_out, reqs) || !in_place(a->n_done, a->n_done_out, reqs))
    return "score_out, tokens_out, length_out and n_done_out must be score, tokens, length and n_done or share no elements with them";
  const long long done = reqs * a->max_done * (a->tokens ? a->capacity : 0);
  if (!apart(a->done_tokens, a->tokens, done, text) || !apart(a->done_tokens, a->tokens_out, done, text))
    return "done_tokens must share no elements with tokens and tokens_out";
  return nullptr;
}

// What one request's threads write must not be what others read or write.
const char* check_beam_apart(const ws_beam_args* a) {
  const long long rows = 4ll * a->n * a->beams, reqs = 4ll * a->n, text = a->tokens ? rows * a->capacity : 0;
  const long long done = reqs * a->max_done;
  struct Array { const void* p; long long bytes; const void* in; };          // in: what it may take the place of
  const Array outs[] = {{a->score_out, rows, a->score}, {a->parent, rows, nullptr}, {a->token, rows, nullptr},
                        {a->tokens_out, text, a->tokens}, {a->length_out, reqs, a->length}, {a->n_done_out, reqs, a->n_done},
                        {a->done_score, done, nullptr}, {a->done_length, done, nullptr},
                        {a->done_tokens, a->tokens ? done * a->capacity : 0, nullptr}};
  for (const Array& x : outs)
    for (const Array& y : outs)
      if (&x != &y && (!apart(x.p, y.p, x.bytes, y.bytes) || !apart(x.p, y.in, x.bytes, y.bytes)))
        return "outputs must share no elements with each other, nor with inputs other than their own";
  return nullptr;
}

struct Plan { int parts, part; size_t stat, bytes; };
// Ten CTAs of 128 threads run on an SM (44 and 46 registers): as many parts as
// fill that round (a row is read once whatever they are), none longer than 256
// logits per thread, and none shorter than four.  480 rows of 51,866: 3 parts
// 33 us.  Parts for twelve CTAs ran into a second round (5 beams over and over on
// the same logits of 16 / 32 / 64 requests: 19.0 / 20.8 / 23.9 us, and 17.7 /
// 18.7 / 22.1 in this form), and registers for twelve spill (18.5 / 20.5 / 24.2).
constexpr int BM_RESIDENT = 10;
Plan make_plan(const ws_beam_args& a) {
  Plan q = {};
  const long long rows = (long long)a.n * a.beams;
  const int least = (a.vocab + BM_PART - 1) / BM_PART, most = min(BM_PARTS, (a.vocab + 4 * BM_NT - 1) / (4 * BM_NT));
  const int want = max(least, (int)min((long long)most, (long long)BM_RESIDENT * SMS / rows));
  q.part = ((a.vocab + want - 1) / want + BM_STEP - 1) / BM_STEP * BM_STEP;
  q.parts = (a.vocab + q.part - 1) / q.part;
  q.stat = (size_t)rows * q.parts * (a.beams + 1) * 8;
  q.bytes = (q.stat + (size_t)rows * q.parts * 8 + 255) / 256 * 256;
  return q;
}

}  // namespace

extern "C" size_t ws_beam_select_workspace(const ws_beam_args* args) {
  return check_beam(args) || args->n == 0 ? 0 : make_plan(*args).bytes;
}

extern "C" int ws_beam_select(const ws_beam_args* args, void* workspace, size_t workspace_bytes, ws_stream stream) {
  if (const char* e = check_beam(args)) return fail(WS_EINVAL, e);
  if (args->n == 0) return WS_OK;
  if (const char* e = check_beam_apart(args)) return fail(WS_EINVAL, e);
  const Plan q = make_plan(*args);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)) return fail(WS_EINVAL, "workspace must be 16-byte aligned and not null");
  if (q.bytes > workspace_bytes) return fail(WS_ENOSPACE, "workspace smaller than ws_beam_select_workspace()");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return fail(WS_ECUDA, (std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior)).c_str());
  BeamP p = {};
  p.a = *args;
  p.parts = q.parts;
  p.part = q.part;
  p.cand = (unsigned long long*)workspace;
  p.stat = (float2*)((char*)workspace + q.stat);
  const cudaStream_t s = (cudaStream_t)stream;
  const size_t list = (size_t)(args->beams + 1) * (q.part / BM_NT) * 8;      // at most 34 KB
  const dim3 grid((unsigned)q.parts, (unsigned)(args->n * args->beams));
  if (((reinterpret_cast<uintptr_t>(args->logits) >> 2) | (uint64_t)args->ld) & 1) scan_kernel<false><<<grid, BM_NT, list, s>>>(p);
  else scan_kernel<true><<<grid, BM_NT, list, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
    ws_count_launches(1);
    const size_t smem = (size_t)args->beams * q.parts * (args->beams + 1) * 8;
    e = cudaFuncSetAttribute(merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BM_BEAMS * BM_PARTS * BM_K * 8);
    if (e == cudaSuccess) e = launch_after(merge_kernel, dim3((unsigned)args->n), BM_MT, smem, s, p);
  }
  if (e != cudaSuccess) return fail(WS_ECUDA, (std::string("beam selection launch: ") + cudaGetErrorString(e)).c_str());
  return WS_OK;
}

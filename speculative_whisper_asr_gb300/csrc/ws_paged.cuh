// Shared by the operators on a caller's paged key/value cache: argument
// checks and the address of a position.
#pragma once
#include <limits.h>
#include <math.h>

#include <string>

#include "ws_internal.cuh"

// Message of a bad cache description, or null.
inline const char* check_paged_cache(const ws_paged_cache* c) {
  if (!c) return "null cache";
  if (c->dtype != WS_F32 && c->dtype != WS_BF16) return "dtype must be WS_F32 or WS_BF16";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535) return "n_kv_heads must be 1..65535";
  if (c->page_size < 1) return "page_size must be >= 1";
  if (c->n_pages < 1) return "n_pages must be >= 1";
  if (!c->k || !c->v || !c->page_table) return "null keys, values or page table";
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15)
    return "keys and values must be 16-byte aligned";
  const int64_t unit = c->dtype == WS_BF16 ? 8 : 4;
  if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < 0 || c->page_stride % unit ||
      c->head_stride % unit || c->token_stride % unit)
    return "cache strides must be multiples of 16 bytes and not negative";
  // the copy engine's strides end at 2^40 bytes
  const int64_t most = (int64_t)1 << 37;
  if (c->page_stride >= most || c->head_stride >= most || c->token_stride >= most) return "cache strides too large";
  if ((c->page_size > 1 && c->token_stride < WS_DH) || (c->n_kv_heads > 1 && c->head_stride < WS_DH) ||
      (c->n_pages > 1 && c->page_stride < WS_DH))
    return "cache strides must be >= 64 elements";
  if (c->n_slots < 1 || c->table_stride < 1) return "n_slots and table_stride must be >= 1";
  return nullptr;
}

inline int paged_fail(int code, const std::string& msg) {
  ws_set_thread_error(msg.c_str());
  return code;
}

// Launch of a kernel whose every thread calls pdl_wait() before it returns: on
// created streams it may start while the kernel before it (which calls
// pdl_trigger()) still runs, as elsewhere in the library.  If all its CTAs left
// without the wait, its end, which the next node of a graph depends on, could
// come before the end of the kernel before it.
template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = s != nullptr && s != cudaStreamLegacy && s != cudaStreamPerThread ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
  if (e == cudaSuccess) ws_count_launches(1);
  return e;
}

// Page of position j of a slot, or -1 where it may not be read.
__device__ __forceinline__ int paged_page(const ws_paged_cache& c, const int32_t* table, int stride, int slot, int j) {
  const int p = j / c.page_size;
  if (p >= stride) return -1;
  const int page = __ldg(table + (size_t)slot * stride + p);
  return page >= 0 && page < c.n_pages ? page : -1;
}
// Element offset of (page, head, position j).
__device__ __forceinline__ size_t paged_off(const ws_paged_cache& c, int page, int head, int j) {
  return (size_t)page * (size_t)c.page_stride + (size_t)head * (size_t)c.head_stride +
         (size_t)(j % c.page_size) * (size_t)c.token_stride;
}

// sv_kv.cu -- the paged cache's bookkeeping and writes: spec_kv_slots,
// spec_kv_append.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "spec_tree.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

// ------------------------------------------------------------------- slots
constexpr int kSThreads = 1024;
constexpr int kRowsCached = 4096;  // requests whose row bounds a block keeps on chip

struct SlotParams {
  const int32_t *lens, *add, *cu, *path;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t *slots, *start, *out_lens, *out_count;
  int64_t table_row;
  int path_width, table_width, pool, B, N, page;
};

struct Request {
  int len, add, have, need;
  bool grows, release;
};

// Request r as its inputs describe it: `grows` when nothing but a lack of
// free pages can refuse it.
__device__ __forceinline__ Request request_of(const SlotParams& P, int r) {
  Request q{};
  q.len = P.lens[r];
  q.add = P.add[r];
  const int lo = P.cu[r], hi = P.cu[r + 1];
  const int64_t cap = static_cast<int64_t>(P.table_width) * P.page;
  bool bad = q.len < 0 || q.len > cap || q.add < -1 || lo < 0 || hi > P.N || hi < lo;
  if (bad) return q;
  q.have = (q.len + P.page - 1LL) / P.page;
  q.release = q.add == -1;
  if (q.release) return q;
  if (q.add > hi - lo || static_cast<int64_t>(q.len) + q.add > cap) return q;
  if (P.path) {
    if (q.add > P.path_width) return q;
    const int32_t* path = P.path + static_cast<size_t>(r) * P.path_width;
    int prev = -1;
    for (int i = 0; i < q.add; ++i) {
      const int x = path[i];
      bad |= x <= prev || x >= hi - lo;
      prev = x;
    }
    if (bad) return q;
  }
  q.grows = true;
  q.need = static_cast<int>((static_cast<int64_t>(q.len) + q.add + P.page - 1) / P.page) - q.have;
  return q;
}

// Inclusive prefix sum over the block; `total` is the block's.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warps, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warps[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += warps[warp - 1];
  total = warps[31];
  return v;
}

// First index in [0, n) whose inclusive prefix exceeds k.
__device__ __forceinline__ int owner_of(const int64_t* incl, int n, int64_t k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > k) {
      hi = mid;
    } else {
      lo = mid + 1;
    }
  }
  return lo;
}

// The last request whose rows start at or before `row`.
__device__ __forceinline__ int request_at(const int32_t* cu, int B, int row) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= row) {
      lo = mid;
    } else {
      hi = mid - 1;
    }
  }
  return lo;
}

// Slot of row `row` if it belongs to request b, -1 when it is not kept.
__device__ __forceinline__ int slot_of(const SlotParams& P, int b, int row) {
  const int first = P.cu[b];
  if (row < first || row >= P.cu[b + 1]) return -1;
  const int begin = P.start[b];
  if (begin < 0) return -1;
  const int add = P.add[b];
  int i = row - first;
  if (P.path) {
    const int32_t* path = P.path + static_cast<size_t>(b) * P.path_width;
    int j = 0;
    while (j < add && path[j] < i) ++j;
    if (j == add || path[j] != i) return -1;
    i = j;
  } else if (i >= add) {
    return -1;
  }
  const int64_t pos = static_cast<int64_t>(begin) + i;
  const int page = P.table[b * P.table_row + pos / P.page];
  const int64_t slot = static_cast<int64_t>(page) * P.page + pos % P.page;
  return page < 0 || slot > INT_MAX ? -1 : static_cast<int>(slot);
}

// The requests' prefix sums decide who grows and which free pages it takes;
// the pages are handed out flat over the threads (a long prompt takes
// thousands).  Bound by latency: one block does it all, slots included, when
// there are few rows.  For many, a cluster of kSlotCtas blocks shares out the
// pages (every block runs the same sums; the first one writes the requests'
// outputs, which may be their inputs, once all have read), and
// slots_rows_kernel does the rows: 512 prompts, 10^6 rows and 66,000 pages
// took 67 us with one block, and take 20.  The border is where one block's time
// reaches that of a call from Python (device, call): 64 requests, 1,024 rows 6.4,
// 19 us with one block, 9.4, 20 with the cluster; 8,192 rows 13.7, 18 and 9.5, 20;
// 16,384 rows 22, 23 and 9.6, 20.
constexpr int kSlotCtas = 8;
template <bool kMany>
__global__ void __launch_bounds__(kSThreads) slots_kernel(const SlotParams P) {
  __shared__ int64_t warps[32];
  __shared__ int64_t incl_s[kSThreads];
  __shared__ int have_s[kSThreads], need_s[kSThreads];
  __shared__ int64_t popped_s;
  __shared__ int release_s;
  const int tid = threadIdx.x;
  const int rank = kMany ? blockIdx.x : 0, ctas = kMany ? kSlotCtas : 1;
  auto sync = [&]() {
    if constexpr (kMany) {
      asm volatile("barrier.cluster.arrive.release;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  const int64_t count = min(max(*P.free_count, 0), P.pool);
  if (tid == 0) {
    popped_s = 0;
    release_s = 0;
  }
  __syncthreads();

  int64_t carry = 0;  // pages asked for by the requests before this round's
  for (int base = 0; base < P.B; base += kSThreads) {
    const int r = base + tid;
    Request q{};
    if (r < P.B) q = request_of(P, r);
    int64_t total;
    const int64_t incl = carry + block_scan(q.need, warps, total);
    const bool ok = q.grows && (q.need == 0 || incl <= count);
    incl_s[tid] = incl;
    have_s[tid] = q.have;
    need_s[tid] = q.need;
    if (q.release) release_s = 1;
    // the largest prefix that still fits (a later one never does)
    if (ok && q.need) atomicMax(reinterpret_cast<unsigned long long*>(&popped_s), static_cast<unsigned long long>(incl));
    sync();
    if (r < P.B && rank == 0) {
      P.start[r] = ok ? q.len : -1;
      if (!q.release) P.out_lens[r] = ok ? q.len + q.add : q.len;
    }
    const int64_t popped = popped_s;
#pragma unroll 4
    for (int64_t k = carry + rank * kSThreads + tid; k < popped; k += ctas * kSThreads) {
      const int o = owner_of(incl_s, kSThreads, k);
      const int64_t nth = k - (incl_s[o] - need_s[o]);
      P.table[(base + o) * P.table_row + have_s[o] + nth] = __ldcg(P.free_pages + (count - 1 - k));
    }
    carry += total;
    __syncthreads();
  }

  int64_t top = count - popped_s;
  sync();  // pages on the stack are overwritten only now
  if (rank != 0) return;
  if (release_s) {  // the pages of released requests go on top of what is left
    for (int base = 0; base < P.B; base += kSThreads) {
      const int r = base + tid;
      Request q{};
      if (r < P.B) q = request_of(P, r);
      const int give = q.release ? q.have : 0;
      int64_t total;
      incl_s[tid] = block_scan(give, warps, total);
      need_s[tid] = give;
      if (q.release) P.out_lens[r] = 0;
      __syncthreads();
      for (int64_t k = tid; k < total; k += kSThreads) {
        const int o = owner_of(incl_s, kSThreads, k);
        const int64_t nth = k - (incl_s[o] - need_s[o]);
        if (top + k < P.pool) P.free_pages[top + k] = P.table[(base + o) * P.table_row + nth];
      }
      top += total;
      __syncthreads();
    }
  }
  if (tid == 0) *P.out_count = static_cast<int>(min(top, static_cast<int64_t>(P.pool)));
  if constexpr (!kMany) {
    __syncthreads();
    for (int row = tid; row < P.N; row += kSThreads) P.slots[row] = P.B ? slot_of(P, request_at(P.cu, P.B, row), row) : -1;
  }
}

// Four consecutive rows a thread: one search, then forward from there.
__global__ void __launch_bounds__(256) slots_rows_kernel(const SlotParams P) {
  __shared__ int32_t bounds[kRowsCached];
  const bool cached = P.B <= kRowsCached;
  if (cached)
    for (int i = threadIdx.x; i < P.B; i += 256) bounds[i] = P.cu[i];
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (row0 >= P.N) return;
  int b = P.B ? request_at(cached ? bounds : P.cu, P.B, static_cast<int>(row0)) : 0;
  int y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = static_cast<int>(min(row0 + i, static_cast<int64_t>(P.N) - 1));
    while (b + 1 < P.B && P.cu[b + 1] <= row) ++b;
    y[i] = P.B ? slot_of(P, b, row) : -1;
  }
  if (row0 + 4 <= P.N && reinterpret_cast<uintptr_t>(P.slots) % 16 == 0) {
    *reinterpret_cast<int4*>(P.slots + row0) = make_int4(y[0], y[1], y[2], y[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row0 + i < P.N) P.slots[row0 + i] = y[i];
  }
}

// ------------------------------------------------------------------ append
struct AppendParams {
  const char* src[2];
  char* cache[2];
  int64_t src_layer[2], src_row[2], src_head[2];  // bytes
  int64_t cache_layer[2], cache_page[2], cache_token[2], cache_head[2];
  const int32_t* slots;
  int64_t units;  // layers * N
  int64_t nslots;
  int N, H, vecs, page;  // vecs: vectors of one head
};

constexpr int kAThreads = 256;

// A warp copies one (layer, row): its slot, then every lane's vectors of the
// keys and the values, four in flight each.  A pure copy, bound by memory.
template <typename T>
__global__ void __launch_bounds__(kAThreads) append_kernel(const __grid_constant__ AppendParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAThreads / 32);
  const int total = P.H * P.vecs;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kAThreads / 32) + (threadIdx.x >> 5); u < P.units; u += warps) {
    const int64_t layer = u / P.N;
    const int row = static_cast<int>(u - layer * P.N);
    const int64_t slot = P.slots[row];
    if (slot < 0 || slot >= P.nslots) continue;
    const int64_t page = slot / P.page, tok = slot - page * P.page;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const char* s = P.src[w] + layer * P.src_layer[w] + row * P.src_row[w];
      char* d = P.cache[w] + layer * P.cache_layer[w] + page * P.cache_page[w] + tok * P.cache_token[w];
#pragma unroll 4
      for (int i = lane; i < total; i += 32) {
        const int h = i / P.vecs, e = i - h * P.vecs;
        reinterpret_cast<T*>(d + h * P.cache_head[w])[e] = __ldg(reinterpret_cast<const T*>(s + h * P.src_head[w]) + e);
      }
    }
  }
}

template <typename T>
void launch_append(AppendParams p, int head_bytes, cudaStream_t stream) {
  p.vecs = head_bytes / static_cast<int>(sizeof(T));
  const int64_t blocks = (p.units + kAThreads / 32 - 1) / (kAThreads / 32);
  append_kernel<T><<<static_cast<unsigned>(std::min<int64_t>(blocks, sm_count() * 8)), kAThreads, 0, stream>>>(p);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

int spec_kv_slots(const int32_t* lens, const int32_t* add, const int32_t* cu_rows,
                  const int32_t* path, int path_width, int32_t* table, int64_t table_row,
                  int table_width, int32_t* free_pages, int pool, const int32_t* free_count, int B,
                  int N, int page_size, int32_t* out_slots, int32_t* out_start,
                  int32_t* out_lens, int32_t* out_free_count, void* stream) {
  if (B < 0 || B > SV_MAX_BATCH)
    return set_error(SV_ERR_INVALID_ARG, "B must be in [0, %d] (got %d)", SV_MAX_BATCH, B);
  if (N < 0) return set_error(SV_ERR_INVALID_ARG, "N must be >= 0 (got %d)", N);
  if (page_size < 1) return set_error(SV_ERR_INVALID_ARG, "page_size must be >= 1 (got %d)", page_size);
  if (table_width < 0 || pool < 0 || (path && path_width < 0))
    return set_error(SV_ERR_INVALID_ARG, "table_width, pool and path_width must be >= 0");
  if (table_row < table_width)
    return set_error(SV_ERR_INVALID_ARG, "table rows overlap: stride %lld < width %d",
                     static_cast<long long>(table_row), table_width);
  if (!free_count || !out_free_count || (N > 0 && !out_slots) || (pool > 0 && !free_pages) ||
      (B > 0 && (!lens || !add || !cu_rows || !out_start || !out_lens || (table_width > 0 && !table))))
    return set_error(SV_ERR_INVALID_ARG, "NULL input or output pointer");
  const void* all[] = {lens, add, cu_rows, path, table, free_pages, free_count, out_slots, out_start, out_lens, out_free_count};
  for (const void* p : all)
    if (misaligned(p, 4)) return set_error(SV_ERR_INVALID_ARG, "pointers must be aligned to their element size");
  int rc = check_device();
  if (rc != SV_OK) return rc;
  SlotParams p{lens, add, cu_rows, path, table, free_pages, free_count, out_slots, out_start,
               out_lens, out_free_count, table_row, path_width, table_width, pool, B, N, page_size};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N <= 8 * kSThreads) {
    slots_kernel<false><<<1, kSThreads, 0, s>>>(p);
    return check_launch("slots");
  }
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kSlotCtas);
  cfg.blockDim = dim3(kSThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kSlotCtas, 1, 1};
  cudaError_t e = cudaLaunchKernelEx(&cfg, slots_kernel<true>, p);
  if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "slots launch: %s", cudaGetErrorString(e));
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(N) + 1023) / 1024));
  cfg.blockDim = dim3(256);
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  e = cudaLaunchKernelEx(&cfg, slots_rows_kernel, p);
  if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "slots rows launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

int spec_kv_append(const sv_kv_append_args* a, void* stream) {
  if (!a) return set_error(SV_ERR_INVALID_ARG, "args is NULL");
  if (a->layers < 0 || a->N < 0 || a->H < 1 || a->D < 1 || a->num_pages < 0 || a->page_size < 1)
    return set_error(SV_ERR_INVALID_ARG, "sizes out of range (layers %d, N %d, H %d, D %d, num_pages %d, page_size %d)",
                     a->layers, a->N, a->H, a->D, a->num_pages, a->page_size);
  const int es = a->elem_bytes;
  if (es != 1 && es != 2 && es != 4)
    return set_error(SV_ERR_INVALID_ARG, "elem_bytes must be 1, 2 or 4 (got %d)", es);
  if (static_cast<int64_t>(a->H) * a->D * es > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "a row of %d x %d elements is too large", a->H, a->D);
  if (a->layers == 0 || a->N == 0 || a->num_pages == 0) return SV_OK;
  if (!a->slots || !a->src[0] || !a->src[1] || !a->cache[0] || !a->cache[1])
    return set_error(SV_ERR_INVALID_ARG, "NULL input or output pointer");
  if (misaligned(a->slots, 4)) return set_error(SV_ERR_INVALID_ARG, "slots must be 4-byte aligned");
  AppendParams p{};
  uint64_t bits = 16;  // every address and byte stride together: the widest vector they allow
  bool flat = true;
  for (int w = 0; w < 2; ++w) {
    if (misaligned(a->src[w], es) || misaligned(a->cache[w], es))
      return set_error(SV_ERR_INVALID_ARG, "pointers must be aligned to their element size");
    p.src[w] = static_cast<const char*>(a->src[w]);
    p.cache[w] = static_cast<char*>(a->cache[w]);
    const int64_t st[7] = {a->src_layer[w], a->src_row[w], a->src_head[w], a->cache_layer[w],
                           a->cache_page[w], a->cache_token[w], a->cache_head[w]};
    p.src_layer[w] = st[0] * es;
    p.src_row[w] = st[1] * es;
    p.src_head[w] = st[2] * es;
    p.cache_layer[w] = st[3] * es;
    p.cache_page[w] = st[4] * es;
    p.cache_token[w] = st[5] * es;
    p.cache_head[w] = st[6] * es;
    bits |= reinterpret_cast<uintptr_t>(a->src[w]) | reinterpret_cast<uintptr_t>(a->cache[w]);
    for (int i = 0; i < 7; ++i) bits |= static_cast<uint64_t>(st[i] * es);
    flat &= a->H == 1 || (a->src_head[w] == a->D && a->cache_head[w] == a->D);
  }
  p.slots = a->slots;
  p.units = static_cast<int64_t>(a->layers) * a->N;
  p.nslots = static_cast<int64_t>(a->num_pages) * a->page_size;
  p.N = a->N;
  p.page = a->page_size;
  p.H = flat ? 1 : a->H;
  const int head_bytes = a->D * es * (flat ? a->H : 1);
  bits |= static_cast<uint64_t>(head_bytes);
  int rc = check_device();
  if (rc != SV_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (bits & (~bits + 1)) {  // lowest set bit
    case 16: launch_append<uint4>(p, head_bytes, s); break;
    case 8: launch_append<uint2>(p, head_bytes, s); break;
    case 4: launch_append<uint32_t>(p, head_bytes, s); break;
    case 2: launch_append<uint16_t>(p, head_bytes, s); break;
    default: launch_append<uint8_t>(p, head_bytes, s); break;
  }
  return check_launch("append");
}

}  // extern "C"

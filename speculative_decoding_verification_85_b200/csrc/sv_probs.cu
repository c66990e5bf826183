// sv_probs.cu -- verification from given probabilities (spec_verify_probs,
// spec_verify_tree): one thread-block cluster per sequence.
//
// With normalised inputs a decision needs two numbers per candidate; a full
// row is read only where a residual's mass or the final draw needs it.  After
// k rejections at one node the law is max(p - c q, 0) / M (c_0 = 0, M_0 = 1,
// c_{k+1} = c_k + M_k, M_{k+1} = sum max(p - c_{k+1} q, 0)), so each
// rejection costs one sum over the row pair and nothing is written.
//
// The sums: every CTA of the cluster sums its slice of the row in chunks of
// 512 entries, a warp a chunk.  A residual over aligned rows takes two chunks of
// both rows at a time (64 entries a lane in flight); plain rows, unaligned ones
// and a slice's last chunks go one chunk at a time.  The slices' sums are
// exchanged through distributed shared memory, every CTA finds the slice that
// the uniform falls into, and one warp of that CTA walks down its chunk sums and
// one chunk again (from L2).  256 chains of 4 at V = 151936 fp32 take 54 us: 0.83
// of the measured copy bandwidth.  Sums are fp64: the order of addition then
// moves a border by 1e-16 of the mass, so the drawn entry is the one of the
// definition.
#include <cuda_runtime.h>

#include "spec_tree.h"
#include "sv_cluster.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kPThreads = 256;
constexpr int kPWarps = kPThreads / 32;
constexpr int kChunk = 512;  // entries one warp sums at a time
constexpr int kMaxCluster = 8;
constexpr size_t kMaxSmem = 200 * 1024;

struct ProbsParams {
  const void* target;
  const void* draft;  // nullptr: point drafts
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu;
  const float* u;
  const float* ud;
  int tree;  // 0: the chain form
  int N, gamma, width, V;
  int cluster, chunks;  // CTAs of a sequence, chunks of one CTA's slice
  int32_t* accept_len;
  int32_t* out_tokens;
  int32_t* out_path;
};

struct ProbsShared {
  double xsum[2][kMaxCluster];  // the slices' sums, double-buffered
  double c, M;                  // the current law: max(p - c q, 0) / M
  int reduce;                   // the decision waits for the next residual's mass
  int cur, last, acc, ngone;    // current node, last child tried, accepted, rejected point drafts
  int lost;                     // the last of those that had mass, or -1
  int bad, n;
  int64_t trow, drow, t0;  // first target row, draft row, token index
};

// One entry's weight: max(p - c q, 0), NaN kept.
__device__ __forceinline__ double weight(double p, double c, double q) {
  const double w = p - c * q;
  return w < 0.0 ? 0.0 : w;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Entries [v, v + 4 k) of a row as this lane holds them in a chunk: element
// e (0..15) of lane l is entry 128 (e / 4) + 4 l + e % 4 (fp32), or
// 256 (e / 8) + 8 l + e % 8 (bf16).
template <bool kBf16>
__device__ __forceinline__ int chunk_entry(int e, int lane) {
  return kBf16 ? 256 * (e >> 3) + 8 * lane + (e & 7) : 128 * (e >> 2) + 4 * lane + (e & 3);
}

// This lane's 16 entries of the whole chunk starting at entry v of a 16-byte
// aligned row: four (bf16: two) 16-byte loads.
template <bool kBf16>
__device__ __forceinline__ void load_whole(const void* row, int v, int lane, float (&x)[16]) {
  if constexpr (kBf16) {
    const uint4* g = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + v);
    uint4 w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] = __ldg(g + 32 * k + lane);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t r[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[8 * k + 2 * i] = bf16_lo(r[i]);
        x[8 * k + 2 * i + 1] = bf16_hi(r[i]);
      }
    }
  } else {
    const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(row) + v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 w = __ldg(g + 32 * k + lane);
      x[4 * k] = w.x;
      x[4 * k + 1] = w.y;
      x[4 * k + 2] = w.z;
      x[4 * k + 3] = w.w;
    }
  }
}

// The same for any chunk; entries from `end` on are 0.  One that is not whole
// or not aligned is 16 element loads, a warp's consecutive.
template <bool kBf16>
__device__ __forceinline__ void load_chunk(const void* row, int v, int end, int lane, bool vec,
                                           float (&x)[16]) {
  if (vec && v + kChunk <= end) {
    load_whole<kBf16>(row, v, lane, x);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int i = v + chunk_entry<kBf16>(e, lane);
      x[e] = i < end ? logit_at<kBf16>(row, i) : 0.0f;
    }
  }
}

// Shared memory behind ProbsShared: chunk sums [chunks] fp64, then per node
// p, q, u (fp32) and token, parent, path, rejected-token list (int).
template <bool kBf16>
__global__ void __launch_bounds__(kPThreads, 3) probs_kernel(const __grid_constant__ ProbsParams P) {
  extern __shared__ __align__(16) char smem[];
  __shared__ ProbsShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % P.cluster, b = blockIdx.x / P.cluster;
  const bool chain = P.tree == 0;
  const bool rows = P.draft != nullptr;
  const int cap = chain ? P.gamma + 1 : min(P.width, SV_MAX_NODES);
  double* csum = reinterpret_cast<double*>(smem);
  float* np = reinterpret_cast<float*>(csum + P.chunks);
  float* nq = np + cap;
  float* nu = nq + cap;
  int* ntok = reinterpret_cast<int*>(nu + cap);
  int* npar = ntok + cap;
  int* npath = npar + cap;
  int* gone = npath + cap;

  // the peers' shared memory may be written once they have started: arrive
  // here, wait before the first exchange
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  if (tid == 0) {
    int n;
    if (chain) {
      n = P.gamma + 1;
      sh.trow = static_cast<int64_t>(b) * n;
      sh.drow = static_cast<int64_t>(b) * P.gamma;
      sh.t0 = sh.drow - 1;  // node i's token and uniform sit at t0 + i
      sh.bad = 0;
    } else {
      const int lo = P.cu[b], hi = P.cu[b + 1];
      n = hi - lo;
      sh.bad = lo < 0 || hi > P.N || n < 1 || n > cap;
      if (sh.bad) n = 0;
      sh.trow = sh.drow = sh.t0 = lo;
    }
    sh.n = n;
    sh.cur = 0;
    sh.last = 0;
    sh.acc = 0;
    sh.ngone = 0;
    sh.lost = -1;
    sh.c = 0.0;
    sh.M = 1.0;
  }
  __syncthreads();
  const int n = sh.n;
  const int64_t trow = sh.trow, drow = sh.drow, t0 = sh.t0;
  const size_t es = kBf16 ? 2 : 4;
  const char* tgt = static_cast<const char*>(P.target);
  const char* drf = static_cast<const char*>(P.draft);
  const size_t rowbytes = static_cast<size_t>(P.V) * es;

  // every node's probabilities at its parent's rows, and the checks
  bool bad = false;
  for (int i = tid; i < n; i += kPThreads) {
    const int par = chain ? i - 1 : P.parents[t0 + i];
    if (i == 0) {
      bad |= par != -1;
      npar[0] = -1;
      continue;
    }
    const int x = P.tokens[t0 + i];
    const float u = P.u[t0 + i];
    float p = 0.0f, q = 1.0f;
    if (par < 0 || par >= i || x < 0 || x >= P.V) {
      bad = true;
    } else {
      p = logit_at<kBf16>(tgt + (trow + par) * rowbytes, x);
      if (rows) q = logit_at<kBf16>(drf + (drow + par) * rowbytes, x);
      bad |= !(p >= 0.0f && p < INFINITY && q >= 0.0f && q < INFINITY);
    }
    bad |= !(u >= 0.0f && u < 1.0f);
    np[i] = p;
    nq[i] = q;
    nu[i] = u;
    ntok[i] = x;
    npar[i] = par;
  }
  const float ud = P.ud[b];
  bad |= !(ud >= 0.0f && ud < 1.0f);
  if (bad) sh.bad = 1;
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");

  const int C = P.cluster;
  const int v0 = static_cast<int>(min(static_cast<int64_t>(rank) * P.chunks * kChunk, static_cast<int64_t>(P.V)));
  const int v1 = static_cast<int>(min(static_cast<int64_t>(rank + 1) * P.chunks * kChunk, static_cast<int64_t>(P.V)));
  int phase = 0;  // exchanges done

  // This lane's 16 weights max(p - c q, 0) of the chunk at v (c == 0: the
  // target row, without the entries of rejected point drafts).
  auto chunk_weights = [&](int cur, double c, int ngone, int v, double(&w)[16]) {
    const char* pr = tgt + (trow + cur) * rowbytes;
    const bool useq = c != 0.0;
    const char* qr = useq ? drf + (drow + cur) * rowbytes : pr;
    const bool vec = reinterpret_cast<uintptr_t>(pr) % 16 == 0 && reinterpret_cast<uintptr_t>(qr) % 16 == 0;
    float p[16];
    load_chunk<kBf16>(pr, v, v1, lane, vec, p);
    if (useq) {
      float q[16];
      load_chunk<kBf16>(qr, v, v1, lane, vec, q);
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = weight(p[e], c, q[e]);
    } else {
      for (int g = 0; g < ngone; ++g) {
        const int at = gone[g] - v;
        if (at >= 0 && at < kChunk) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (chunk_entry<kBf16>(e, lane) == at) p[e] = 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = weight(p[e], 0.0, 0.0);
    }
  };

  // The mass of that law over the whole row: chunk sums into csum, the
  // slices' sums into every CTA's xsum.  The same bits in every CTA.
  auto reduce = [&](int cur, double c, int ngone) {
    // Whole chunks of aligned row pairs, two of them at a time, all loads first: a CTA that has a
    // row pair to itself is bound by what it has in flight.
    const char* pr = tgt + (trow + cur) * rowbytes;
    const char* qr = c != 0.0 ? drf + (drow + cur) * rowbytes : pr;
    const bool vec = c != 0.0 && reinterpret_cast<uintptr_t>(pr) % 16 == 0 && reinterpret_cast<uintptr_t>(qr) % 16 == 0;
    int k = warp;
    for (; vec && v0 + (k + kPWarps + 1) * kChunk <= v1; k += 2 * kPWarps) {
      float p[2][16], q[2][16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        load_whole<kBf16>(pr, v0 + (k + i * kPWarps) * kChunk, lane, p[i]);
        load_whole<kBf16>(qr, v0 + (k + i * kPWarps) * kChunk, lane, q[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        double s = 0.0;
#pragma unroll
        for (int e = 0; e < 16; ++e) s += weight(p[i][e], c, q[i][e]);
        s = warp_sum(s);
        if (lane == 0) csum[k + i * kPWarps] = s;
      }
    }
    for (; k < P.chunks; k += kPWarps) {
      const int v = v0 + k * kChunk;
      double s = 0.0;
      if (v < v1) {
        double w[16];
        chunk_weights(cur, c, ngone, v, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) s += w[e];
        s = warp_sum(s);
      }
      if (lane == 0) csum[k] = s;
    }
    __syncthreads();
    if (warp == 0) {
      double s = 0.0;
      for (int k = lane; k < P.chunks; k += 32) s += csum[k];
      s = warp_sum(s);
      if (lane < C)
        asm volatile("st.shared::cluster.f64 [%0], %1;"
                     ::"r"(mapa(&sh.xsum[phase & 1][rank], lane)), "d"(s) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    double total = 0.0;
    for (int r = 0; r < C; ++r) total += sh.xsum[phase & 1][r];
    ++phase;
    return total;
  };

  // Decisions, taken by warp 0 of every CTA alike (the same data in the same
  // order), until one needs a residual's mass or no child is left.
  bool ok = sh.bad == 0;
  int held = -1;  // node whose current law csum and xsum hold
  int cur = 0;
  double total = 0.0;
  int only = -1;  // the token to draw where the rejected point drafts left no mass
  while (ok) {
    if (warp == 0) {
      int at = sh.cur, last = sh.last, acc = sh.acc, ngone = sh.ngone, lost = sh.lost, need = 0;
      double c = sh.c, M = sh.M;
      for (;;) {
        int child = n;
        for (int base = last + 1; base < n && child == n; base += 32) {
          const int i = base + lane;
          const unsigned hit = __ballot_sync(0xffffffffu, i < n && npar[i] == at);
          if (hit) child = base + __ffs(hit) - 1;
        }
        if (child == n) break;
        last = child;
        const double p = np[child], u = nu[child];
        bool yes;
        if (rows) {
          const double q = nq[child];
          yes = u * q * M < weight(p, c, q);
        } else {
          double left = p;  // 0 once the token was rejected here
          for (int g = 0; g < ngone; ++g)
            if (gone[g] == ntok[child]) left = 0.0;
          yes = u * M < left;
          if (!yes) {
            M -= left;
            if (left > 0.0) lost = ntok[child];
            if (lane == 0) gone[ngone] = ntok[child];
            __syncwarp();
            ++ngone;
          }
        }
        if (yes) {
          at = child;
          c = 0.0;
          M = 1.0;
          ngone = 0;
          lost = -1;
          if (lane == 0) npath[acc] = child;
          ++acc;
        } else if (rows) {
          need = 1;
          break;
        }
      }
      if (lane == 0) {
        sh.cur = at;
        sh.last = last;
        sh.acc = acc;
        sh.ngone = ngone;
        sh.lost = lost;
        sh.c = c;
        sh.M = M;
        sh.reduce = need;
      }
    }
    __syncthreads();
    cur = sh.cur;
    if (sh.reduce) {
      const double c = sh.c + sh.M;
      const double m = reduce(cur, c, 0);  // (its barriers order the reads above)
      ok = m >= 0.0 && m < INFINITY;
      if (m > 0.0) {
        held = cur;
        total = m;
        if (tid == 0) {
          sh.c = c;
          sh.M = m;
        }
      } else {
        held = -1;  // no mass: the law stays as it was
      }
      __syncthreads();
      continue;
    }
    if (held != cur) total = reduce(cur, sh.c, sh.ngone);
    if (total == 0.0) only = sh.lost;
    ok = only >= 0 || (total > 0.0 && total < INFINITY);
    break;
  }

  const int acc = ok ? sh.acc : -1;
  if (rank == 0) {
    int32_t* otok = P.out_tokens + static_cast<size_t>(b) * P.width;
    for (int i = tid; i < P.width; i += kPThreads)
      if (i != acc) otok[i] = i < acc ? ntok[npath[i]] : -1;
    if (P.out_path) {
      int32_t* opath = P.out_path + static_cast<size_t>(b) * P.width;
      for (int i = tid; i < P.width; i += kPThreads)
        opath[i] = i > acc ? -1 : (i == 0 ? 0 : npath[i - 1]);
    }
    if (tid == 0) {
      P.accept_len[b] = acc;
      if (only >= 0) otok[acc] = only;
    }
  }
  if (!ok || only >= 0) return;

  // The draw: the first entry whose cumulative weight exceeds t.  (Sums of
  // the same weights in another order may differ by a rounding: where that
  // leaves none beyond t, the last entry with weight is the one.)
  const double t = static_cast<double>(ud) * total;
  const double* xs = sh.xsum[(phase - 1) & 1];
  double pre = 0.0, run = 0.0;
  int win = -1;
  for (int r = 0; r < C; ++r) {
    if (xs[r] > 0.0 && !(win >= 0 && pre + xs[win] > t)) {
      win = r;
      pre = run;
    }
    run += xs[r];
  }
  if (rank != win || warp != 0) return;
  const double c = sh.c;
  const int ngone = sh.ngone;
  int chunk = -1;
  double before = 0.0;  // weight before the chosen chunk
  bool found = false;
  run = pre;
  for (int base = 0; base < P.chunks && !found; base += 32) {
    const double s = base + lane < P.chunks ? csum[base + lane] : 0.0;
    double incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned over = __ballot_sync(0xffffffffu, s > 0.0 && run + incl > t);
    const unsigned some = __ballot_sync(0xffffffffu, s > 0.0);
    const int l = over ? __ffs(over) - 1 : (some ? 31 - __clz(some) : -1);
    if (l >= 0) {
      chunk = base + l;
      before = run + __shfl_sync(0xffffffffu, incl - s, l);
      found = over != 0;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  const int v = v0 + chunk * kChunk;
  double w[16];
  chunk_weights(cur, c, ngone, v, w);
  constexpr int kRun = kBf16 ? 8 : 4;  // consecutive entries of a lane
  int best = -1, lastpos = -1;
  run = before;
#pragma unroll
  for (int k = 0; k < 16 / kRun; ++k) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      s += w[k * kRun + i];
      if (w[k * kRun + i] > 0.0) lastpos = chunk_entry<kBf16>(k * kRun + i, lane);
    }
    double incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned over = __ballot_sync(0xffffffffu, s > 0.0 && run + incl > t);
    if (over && best < 0) {
      const int l = __ffs(over) - 1;
      double r2 = run + (incl - s);
      int at = -1;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const double wi = w[k * kRun + i];
        const bool done = at >= 0 && r2 > t;
        if (!done && wi > 0.0) {
          at = chunk_entry<kBf16>(k * kRun + i, lane);
          r2 += wi;
        }
      }
      best = __shfl_sync(0xffffffffu, at, l);
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lastpos = max(lastpos, __shfl_xor_sync(0xffffffffu, lastpos, o));
  if (best < 0) best = lastpos;
  if (lane == 0) P.out_tokens[static_cast<size_t>(b) * P.width + acc] = v + best;
}

template <bool kBf16>
int launch_probs(ProbsParams p, int B, cudaStream_t stream) {
  const int nch = static_cast<int>((static_cast<int64_t>(p.V) + kChunk - 1) / kChunk);
  // Cluster size: as many CTAs as run at once (three a SM), so that none waits for a second
  // wave; trees with draft laws, which take sum after sum from the same rows, gain from more
  // CTAs even so.  No slice is below one chunk a warp.  (V = 151936 fp32 chains: 64 sequences
  // 20 us with four CTAs each, 25 with eight; 128: 30 with two, 37 with four; 256: 53 with one,
  // 61 with two.  V = 128256 bf16 trees of 21 nodes: 64 sequences 31 us with eight, 32 with four,
  // 45 with two.)
  const int limit = (p.tree && p.draft ? 8 : 3) * sm_count();
  int C = 1;
  while (C < kMaxCluster && B * C * 2 <= limit && nch > C * kPWarps) C *= 2;
  p.cluster = C;
  p.chunks = (nch + C - 1) / C;
  const int cap = p.tree ? (p.width < SV_MAX_NODES ? p.width : SV_MAX_NODES) : p.gamma + 1;
  const size_t smem = static_cast<size_t>(p.chunks) * sizeof(double) + static_cast<size_t>(cap) * 7 * 4;
  if (smem > kMaxSmem)
    return set_error(SV_ERR_UNSUPPORTED, "V = %d is too large for B = %d", p.V, B);
  const int rc = allow_smem(reinterpret_cast<const void*>(probs_kernel<kBf16>), kMaxSmem);
  if (rc != SV_OK) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * C);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {static_cast<unsigned>(C), 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, probs_kernel<kBf16>, p);
  if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "probs launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

int probs_call(const ProbsParams& p, int B, int dtype, cudaStream_t stream) {
  int rc = check_device();
  if (rc != SV_OK) return rc;
  return dtype == SV_BF16 ? launch_probs<true>(p, B, stream) : launch_probs<false>(p, B, stream);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

int spec_verify_probs(const void* target_probs, const void* draft_probs,
                      const int32_t* draft_tokens, const float* uniforms,
                      const float* draw_uniforms, int B, int gamma, int V, int dtype,
                      int32_t* out_accept_len, int32_t* out_tokens, void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return set_error(SV_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (B < 0 || B > SV_MAX_BATCH)
    return set_error(SV_ERR_INVALID_ARG, "B must be in [0, %d] (got %d)", SV_MAX_BATCH, B);
  if (gamma < 1 || gamma > SV_MAX_GAMMA)
    return set_error(SV_ERR_INVALID_ARG, "draft length must be in [1, %d] (got %d)", SV_MAX_GAMMA, gamma);
  if (V < 1) return set_error(SV_ERR_INVALID_ARG, "V must be >= 1 (got %d)", V);
  if (B == 0) return SV_OK;
  if (!target_probs || !draft_tokens || !uniforms || !draw_uniforms || !out_accept_len || !out_tokens)
    return set_error(SV_ERR_INVALID_ARG, "NULL input or output pointer");
  const size_t es = dtype == SV_BF16 ? 2 : 4;
  if (misaligned(target_probs, es) || misaligned(draft_probs, es) || misaligned(draft_tokens, 4) ||
      misaligned(uniforms, 4) || misaligned(draw_uniforms, 4) || misaligned(out_accept_len, 4) ||
      misaligned(out_tokens, 4))
    return set_error(SV_ERR_INVALID_ARG, "pointers must be aligned to their element size");
  ProbsParams p{};
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = draft_tokens;
  p.u = uniforms;
  p.ud = draw_uniforms;
  p.gamma = gamma;
  p.width = gamma + 1;
  p.V = V;
  p.accept_len = out_accept_len;
  p.out_tokens = out_tokens;
  return probs_call(p, B, dtype, static_cast<cudaStream_t>(stream));
}

int spec_verify_tree(const void* target_probs, const void* draft_probs, const int32_t* tokens,
                     const int32_t* parents, const int32_t* cu_nodes, const float* uniforms,
                     const float* draw_uniforms, int B, int N, int max_nodes, int V, int dtype,
                     int32_t* out_accept_len, int32_t* out_tokens, int32_t* out_path,
                     void* stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return set_error(SV_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (B < 0 || B > SV_MAX_BATCH)
    return set_error(SV_ERR_INVALID_ARG, "B must be in [0, %d] (got %d)", SV_MAX_BATCH, B);
  if (N < 0) return set_error(SV_ERR_INVALID_ARG, "N must be >= 0 (got %d)", N);
  if (max_nodes < 1) return set_error(SV_ERR_INVALID_ARG, "max_nodes must be >= 1 (got %d)", max_nodes);
  if (V < 1) return set_error(SV_ERR_INVALID_ARG, "V must be >= 1 (got %d)", V);
  if (B == 0) return SV_OK;
  if (!cu_nodes || !draw_uniforms || !out_accept_len || !out_tokens ||
      (N > 0 && (!target_probs || !tokens || !parents || !uniforms)))
    return set_error(SV_ERR_INVALID_ARG, "NULL input or output pointer");
  const size_t es = dtype == SV_BF16 ? 2 : 4;
  if (misaligned(target_probs, es) || misaligned(draft_probs, es) || misaligned(tokens, 4) ||
      misaligned(parents, 4) || misaligned(cu_nodes, 4) || misaligned(uniforms, 4) ||
      misaligned(draw_uniforms, 4) || misaligned(out_accept_len, 4) || misaligned(out_tokens, 4) ||
      misaligned(out_path, 4))
    return set_error(SV_ERR_INVALID_ARG, "pointers must be aligned to their element size");
  ProbsParams p{};
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = tokens;
  p.tree = 1;
  p.parents = parents;
  p.cu = cu_nodes;
  p.u = uniforms;
  p.ud = draw_uniforms;
  p.N = N;
  p.width = max_nodes;
  p.V = V;
  p.accept_len = out_accept_len;
  p.out_tokens = out_tokens;
  p.out_path = out_path;
  return probs_call(p, B, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// sv_attn.cu -- spec_tree_attention: softmax attention of drafted nodes over a
// paged context and their own ancestors (tcgen05 + TMA).
//
// Work.  A unit is (sequence, key head, up to two tiles of 128 query rows); a
// row is (node, query head of the key head's group), nodes first, so a tile
// holds 128 / G whole nodes.  A unit's keys are cut into tiles of 128: the
// tree's own (last first, so that every row's walk up its ancestors passes
// them in order), then the context's.  All units' tiles form one line, which
// is cut into equal stretches, one per SM: a ragged batch and one long
// sequence both keep every SM busy.  A unit cut by a border leaves partial
// results (unnormalised output, exponent shift, sum) in the workspace and
// combine_kernel joins them in a fixed order.
//
// One CTA: TMA fills a ring of key and value tiles; one thread issues the
// products S = Q K^T (fp32, tensor memory) and O += P V; two groups of four
// warps turn S into P, a thread a row (maximum, exponentials and sum need no
// exchange).  Products are issued as a sequence of steps that alternate
// between the two groups: with two query tiles both groups take every key
// tile, with one the groups take the key tiles in turn and their results are
// joined at the end (both read the other's accumulator: same lanes).  So one
// group's exponentials always run beside the other's products.  The
// accumulator is rescaled only when a row's maximum has grown by more than
// 2^8; until then weights up to 2^8 are accumulated, exactly as well.
//
// Bound by memory up to about 250 query rows per key head.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "spec_tree.h"
#include "sv_internal.h"
#include "sv_tc.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;          // keys of a tile, rows of a query tile
constexpr int kWarpsSoft = 8;       // softmax warps: two groups of four
constexpr int kSoft = 32 * kWarpsSoft;
constexpr int kWarpK = 8, kWarpV = 9, kWarpMma = 10, kWarpQ = 11;
constexpr int kThreads = 32 * 12;
// Registers: the two softmax groups hold a row of 128 scores a thread, the
// third group needs few.  2 x 208 + 88 = 3 x 168, what a block of 384 threads
// is launched with.
constexpr int kRegsSoft = 208, kRegsRest = 88;
constexpr float kGrow = 8.0f;       // base-2 growth of a maximum that is let stand
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTreeBox = 16;        // rows of one load of the nodes' own keys and values

template <int DP>
struct Shape {
  static constexpr int kHalves = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kStages = DP == 128 ? 5 : 10;
  static constexpr size_t kTiles = static_cast<size_t>(2 + kStages) * kTileBytes;
};

struct alignas(64) AttnParams {
  CUtensorMap qmap, kmap, vmap, kcmap, vcmap;
  void* out;
  float* lse;
  const int32_t *table, *lens, *parents, *cu;
  const uint16_t* v;  // the nodes' own values
  int64_t v_node, v_head, table_row;
  int B, N, Hq, Hkv, G, D, num_pages, page, width;
  int box;             // tokens of one load from a page
  int npt;             // nodes of one query tile
  float sl;            // scale * log2(e)
  float* part_o;       // partial results: [cta][2][tile][DP / 4][128][4]
  float2* part_s;      // [cta][2][tile][128] (shift, sum)
  int4* desc;          // [cta][2]: the unit that a border behind this CTA cuts
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// What one sequence asks for.
struct Seq {
  int lo, n, len, tt, J, U;
  bool mark;
};
__device__ __forceinline__ Seq seq_of(const AttnParams& P, int b) {
  Seq s{};
  s.lo = P.cu[b];
  const int hi = P.cu[b + 1];
  if (s.lo < 0 || hi > P.N || hi <= s.lo) return s;
  s.n = hi - s.lo;
  s.len = P.lens[b];
  s.mark = s.n > SV_MAX_NODES || s.len < 0 || s.len > static_cast<int64_t>(P.width) * P.page;
  if (s.mark) s.len = 0;
  s.tt = cdiv(min(s.n, SV_MAX_NODES), kTile);
  s.J = s.tt + cdiv(s.len, kTile);
  s.U = cdiv(s.n, 2 * P.npt);
  return s;
}

// A CTA's stretch of the line of tiles, unit by unit.
struct Walk {
  int b, hu, j;       // next sequence, unit within it, tile within that
  int64_t left;       // tiles left
  Seq s;
  // the current unit's part
  int h, u, j0, j1;
  bool two;           // two query tiles
  __device__ __forceinline__ bool next(const AttnParams& P) {
    if (left <= 0) return false;
    while (s.n == 0 || hu >= P.Hkv * s.U) {
      ++b;
      hu = 0;
      j = 0;
      s = seq_of(P, b);
    }
    h = hu / s.U;
    u = hu - h * s.U;
    j0 = j;
    j1 = static_cast<int>(min(static_cast<int64_t>(s.J), j0 + left));
    left -= j1 - j0;
    two = s.n - u * 2 * P.npt > P.npt;
    if (j1 == s.J) {
      ++hu;
      j = 0;
    } else {
      j = j1;
    }
    return true;
  }
};

struct Shared {
  uint64_t full[10], empty[10];
  uint64_t qfull[2], qempty[2], sfull[2], pready[2], pvdone[2], oempty, drain;
  float2 xch[2][kTile];
  int64_t scan[16];
  Walk start;
  uint32_t tmem;
  int dead, badv;
};

// Wait for a phase; false once any wait of the CTA has run out of time.
__device__ __forceinline__ bool wait_long(Shared& sh, uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  for (;;) {
    for (int k = 0; k < 64; ++k)
      if (mbar_try_wait(bar, parity)) return true;
    volatile int* dead = &sh.dead;
    if (*dead) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *dead = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity) {
  for (int k = 0; k < 16; ++k)
    if (mbar_try_wait(bar, parity)) return true;
  return wait_long(sh, bar, parity);
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_sync_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(static_cast<uint32_t>(x)) : "memory");
  return r != 0;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  } else {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  }
  return r;
}
// Two fp32 values in one 64-bit register, for the paired instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float pair_lo(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float pair_hi(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <bool kBf16>
constexpr uint32_t kExpMask = kBf16 ? 0x7F80u : 0x7C00u;
template <bool kBf16>
__device__ __forceinline__ bool not_finite(uint32_t half) {
  return (half & kExpMask<kBf16>) == kExpMask<kBf16>;
}
template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t half) {
  if constexpr (kBf16) return __uint_as_float(half << 16);
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<uint16_t>(half)));
  return f;
}

template <int DP, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnParams P) {
  using S = Shape<DP>;
  extern __shared__ __align__(1024) char smem[];
  char* qtile = smem;                           // two query tiles
  char* ring = qtile + 2 * S::kTileBytes;       // key and value tiles in turn
  Shared& sh = *reinterpret_cast<Shared*>(smem + S::kTiles);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qfull[i], 1);
      mbar_init(&sh.qempty[i], 1);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pready[i], kTile);
      mbar_init(&sh.pvdone[i], 1);
    }
    mbar_init(&sh.oempty, kWarpsSoft);
    mbar_init(&sh.drain, 1);
    mbar_init_fence();
    sh.dead = 0;
    sh.badv = 0;
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();

  // ---- where this CTA's stretch begins: prefix sums of the sequences' tiles
  int64_t total = 0, chunk = 0, begin = 0;
  for (int pass = 0; pass < 2; ++pass) {  // the total, then the sequence that `begin` lies in
    int64_t carry = 0;
    for (int base = 0; base < P.B; base += kThreads) {
      const int b = base + tid;
      Seq s{};
      if (b < P.B) s = seq_of(P, b);
      const int64_t mine = static_cast<int64_t>(s.J) * s.U * P.Hkv;
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      __syncthreads();
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      int64_t before = carry;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        carry += sh.scan[w];
      }
      incl += before;
      if (P.B <= kThreads || pass == 1) {
        if (pass == 0) {
          total = carry;
          chunk = (total + gridDim.x - 1) / gridDim.x;
          begin = cta * chunk;
        }
        if (mine > 0 && incl - mine <= begin && begin < incl) {
          Walk w{};
          int64_t at = begin - (incl - mine);
          w.b = b;
          w.s = s;
          w.hu = static_cast<int>(at / s.J);
          w.j = static_cast<int>(at - static_cast<int64_t>(w.hu) * s.J);
          w.left = min(chunk, total - begin);
          sh.start = w;
        }
      }
    }
    if (pass == 0) {
      total = carry;
      chunk = (total + gridDim.x - 1) / gridDim.x;
      begin = cta * chunk;
      if (P.B <= kThreads) break;
    }
  }
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;");
  Walk w{};
  if (begin < total) w = sh.start;  // else nothing is left for this CTA
  const uint32_t tmem = sh.tmem;

  if (warp >= kWarpsSoft) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
  if (warp == kWarpK || warp == kWarpV) {
    // ---------------------------------------------------- keys and values
    // one warp each: ring positions 2 t (keys of the CTA's tile t) and 2 t + 1 (its values)
    const bool kv = warp == kWarpV;
    const CUtensorMap* own = kv ? &P.vmap : &P.kmap;
    const CUtensorMap* cached = kv ? &P.vcmap : &P.kcmap;
    int st = kv ? 1 : 0, ph = 1, t = 0;  // stage, parity of its last release, tiles begun
    bool ok = true;
    while (ok && w.next(P)) {
      const int32_t* row = P.table + w.b * P.table_row;
      // this lane's page of the next context tile, read a tile ahead
      auto page_at = [&](int j) {
        if (j < w.s.tt || j >= w.j1) return 0;
        const int tok = (j - w.s.tt) * kTile + lane * P.box;
        return lane < kTile / P.box && tok < w.s.len ? row[tok / P.page] : 0;
      };
      int page = page_at(w.j0);
      for (int j = w.j0; j < w.j1; ++j) {
        const int ahead = page_at(j + 1);
        const bool tree = j < w.s.tt;
        const int first = tree ? (w.s.tt - 1 - j) * kTile : (j - w.s.tt) * kTile;
        const int valid = min(kTile, (tree ? min(w.s.n, SV_MAX_NODES) : w.s.len) - first);
        const int rows = tree ? kTreeBox : P.box;
        const int boxes = cdiv(valid, rows);
        if (page < 0 || page >= P.num_pages) page = 0;  // (the softmax warps mark the rows)
        ok = __all_sync(0xffffffffu, wait(sh, &sh.empty[st], ph));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], boxes * rows * 128 * S::kHalves);
        __syncwarp();
        if (lane < boxes) {
          char* dst = ring + st * S::kTileBytes + lane * rows * 128;
          if (tree) {
#pragma unroll
            for (int hf = 0; hf < S::kHalves; ++hf)
              tma_3d(dst + hf * (kTile * 128), own, hf * 64, w.h, w.s.lo + first + lane * kTreeBox, &sh.full[st]);
          } else {
            const int tok = P.box == kTile ? first % P.page : 0;
#pragma unroll
            for (int hf = 0; hf < S::kHalves; ++hf)
              tma_4d(dst + hf * (kTile * 128), cached, hf * 64, tok, w.h, page, &sh.full[st]);
          }
        }
        __syncwarp();
        page = ahead;
        ++t;
        if ((st += 2) >= S::kStages) {
          st -= S::kStages;
          ph ^= 1;
        }
      }
    }
    if (!ok) {  // leave no copy in flight behind
      for (int i = max(0, t - S::kStages); i < t; ++i) {
        const int pos = 2 * i + (kv ? 1 : 0);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(&sh.full[pos % S::kStages], (pos / S::kStages) & 1) && global_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == kWarpQ) {
    // ------------------------------------------------------------ queries
    if (lane == 0) {
      int q = 0;  // query tiles loaded
      bool ok = true;
      while (ok && w.next(P)) {
        for (int i = 0; ok && i < (w.two ? 2 : 1); ++i, ++q) {
          const int st = q & 1, use = q >> 1;
          if (use > 0 && !wait(sh, &sh.qempty[st], (use - 1) & 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sh.qfull[st], P.npt * P.G * 128 * S::kHalves);
          for (int hf = 0; hf < S::kHalves; ++hf)
            tma_3d(qtile + st * S::kTileBytes + hf * (kTile * 128), &P.qmap, hf * 64, w.h * P.G,
                   w.s.lo + (w.u * 2 + i) * P.npt, &sh.qfull[st]);
        }
      }
      if (!ok) {
        for (int i = max(0, q - 2); i < q; ++i) {
          const uint64_t t0 = global_ns();
          while (!mbar_try_wait(&sh.qfull[i & 1], (i >> 1) & 1) && global_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // ----------------------------------------------------------- products
    // (the whole warp keeps the books, one lane issues)
    const bool issuer = elect_one();
    constexpr uint32_t idesc_s = instr_desc(kBf16, kTile, false);
    constexpr uint32_t idesc_o = instr_desc(kBf16, DP, true);
    constexpr int kStep = S::kTileBytes >> 4;  // from one tile's descriptor to the next's
    const int ksteps = cdiv(P.D, 16);
    const uint64_t qdesc = smem_desc(smem_addr(qtile), 16);
    const uint64_t kdesc = smem_desc(smem_addr(ring), 16);
    const uint64_t vdesc = smem_desc(smem_addr(ring), kTile * 128);
    int kst = 0, kph = 0, vst = 1, vph = 0;  // next key and value tile: stage, parity
    int q0 = 0, seg = 0;                     // query tiles and parts so far
    uint32_t npv[2] = {0, 0};                // second products so far, by group
    bool ok = true;
    while (ok && w.next(P)) {
      const int T = w.j1 - w.j0;
      const bool two = w.two;
      const int steps = two ? 2 * T : T;
      // S of group s from the next key tile, once the tensor memory it goes to is free;
      // `last`: the group's last of this part
      auto scores = [&](int s, bool last) {
        const int qs = (q0 + (two ? s : 0)) & 1;
        bool fine = npv[s] == 0 || wait(sh, &sh.pvdone[s], (npv[s] - 1) & 1);
        fine = fine && ((two && s) || wait(sh, &sh.full[kst], kph));
        if (!__all_sync(0xffffffffu, fine)) return false;
        tc_fence_after();
        if (issuer) {
          const uint64_t da = qdesc + qs * kStep, db = kdesc + kst * kStep;
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const int off = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;
            if (k < ksteps) mma_ss(tmem + s * kTile, da + off, db + off, idesc_s, k > 0);
          }
          mma_commit(&sh.sfull[s]);
          if (!two || s) mma_commit(&sh.empty[kst]);
          if (last) mma_commit(&sh.qempty[qs]);
        }
        __syncwarp();
        if (!two || s) {
          if ((kst += 2) >= S::kStages) {
            kst -= S::kStages;
            kph ^= 1;
          }
        }
        return true;
      };
      ok = wait(sh, &sh.qfull[q0 & 1], (q0 >> 1) & 1);
      if (two) ok = ok && wait(sh, &sh.qfull[(q0 + 1) & 1], ((q0 + 1) >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok) && scores(0, T == 1) && (steps < 2 || scores(1, two ? T == 1 : T == 2));
      if (ok && seg > 0) ok = __all_sync(0xffffffffu, wait(sh, &sh.oempty, (seg - 1) & 1));
      for (int i = 0; ok && i < steps; ++i) {
        const int s = i & 1;
        bool fine = (two && s) || wait(sh, &sh.full[vst], vph);
        fine = fine && wait(sh, &sh.pready[s], npv[s] & 1);
        ok = __all_sync(0xffffffffu, fine);
        if (!ok) break;
        tc_fence_after();
        if (issuer) {
          const uint32_t o = tmem + 2 * kTile + s * kTile, p = tmem + s * kTile;
          const uint64_t db = vdesc + vst * kStep;
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) mma_ts(o, p + k * 8, db + k * (2048 >> 4), idesc_o, k > 0 || i >= 2);
          mma_commit(&sh.pvdone[s]);
          if (!two || s) mma_commit(&sh.empty[vst]);
        }
        __syncwarp();
        if (!two || s) {
          if ((vst += 2) >= S::kStages) {
            vst -= S::kStages;
            vph ^= 1;
          }
        }
        if (s) ++npv[1]; else ++npv[0];
        // the last key tile's query tiles are free after it (with one query tile: after step T - 1)
        if (i + 2 < steps) ok = scores(s, two ? i + 4 >= steps : i + 3 == steps);
      }
      q0 += two ? 2 : 1;
      ++seg;
    }
    if (!ok) {  // let the products in flight end
      if (issuer) mma_commit(&sh.drain);
      const uint64_t ts = global_ns();
      while (!mbar_try_wait(&sh.drain, 0) && global_ns() - ts < kWaitLimitNs) {
      }
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int wg = warp >> 2, r = tid & (kTile - 1);
    const int rnode = r / P.G, rg = r - rnode * P.G;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + wg * kTile, o_at = tmem + lanes + 2 * kTile;
    const float sl = P.sl;
    int t0 = 0;                 // ring position
    uint32_t steps_done = 0;    // steps of this group so far
    bool alive = true;
    int dseg = 0;
    float shift = 0.0f, sum = 0.0f;  // this row's exponent shift (base 2) and sum of weights

    // S of one key tile to P: shift, sum and, when a maximum has grown much, the accumulator.
    // kMask: 0 every key counts, 1 the first `valid`, 2 those in `see`.
    auto weigh = [&](auto mask, bool fresh, bool mine, int valid, const uint32_t* see) {
      constexpr int kMask = decltype(mask)::value;
      float x[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld32(s_at + c, x + c);
      tc_wait_ld();
      if constexpr (kMask == 2) {
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (!(see[c >> 5] >> (c & 31) & 1)) x[c] = -INFINITY;
      } else if constexpr (kMask == 1) {
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c >= valid) x[c] = -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < kTile; c += 2) mx[(c >> 1) & 3] = fmaxf(fmaxf(mx[(c >> 1) & 3], x[c]), x[c + 1]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
      if (fresh) {
        shift = top;
      } else if (__any_sync(0xffffffffu, mine && top - shift > kGrow)) {
        const float now = fmaxf(shift, top);
        const float f = now == shift ? 1.0f : ex2_approx(shift - now);
        shift = now;
        sum *= f;
#pragma unroll 1
        for (int c = 0; c < DP; c += 16) {
          float o[16];
          tmem_ld16(o_at + wg * kTile + c, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tmem_st16(o_at + wg * kTile + c, reinterpret_cast<uint32_t*>(o));
        }
      }
      const float neg = shift == -INFINITY ? 0.0f : -shift;
      const uint64_t sl2 = pair(sl, sl), neg2 = pair(neg, neg);
      uint64_t part[2] = {0, 0};
#pragma unroll
      for (int c0 = 0; c0 < kTile; c0 += 32) {
        // weights rounded to the input type (relative 2^-8 / 2^-11 at most, as the output
        // itself is, and averaged over the keys); the sum takes them unrounded
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const uint64_t y = fma2(pair(x[c0 + c], x[c0 + c + 1]), sl2, neg2);
          const float a = ex2_approx(pair_lo(y)), b = ex2_approx(pair_hi(y));
          part[(c >> 1) & 1] = add2(part[(c >> 1) & 1], pair(a, b));
          pk[c >> 1] = pack2<kBf16>(a, b);
        }
        tmem_st16(s_at + (c0 >> 1), pk);
      }
      const uint64_t p = add2(part[0], part[1]);
      sum += pair_lo(p) + pair_hi(p);
      tc_wait_st();
    };
    while (w.next(P)) {
      const int T = w.j1 - w.j0;
      const int node = w.u * 2 * P.npt + (w.two ? wg * P.npt : 0) + rnode;  // within the sequence
      const bool mine = rnode < P.npt && node < w.s.n;
      const bool busy = __any_sync(0xffffffffu, mine);  // does this warp hold a row at all
      const int32_t* parents = P.parents + w.s.lo;
      // pages outside the cache: this part's rows are marked
      bool bad = w.s.mark;
      if (w.j1 > w.s.tt) {
        const int c0 = max(w.j0 - w.s.tt, 0) * kTile, c1 = min(w.s.len, (w.j1 - w.s.tt) * kTile);
        const int32_t* row = P.table + w.b * P.table_row;
        for (int p = c0 / P.page + tid; p <= (c1 - 1) / P.page; p += kSoft) {
          const int id = row[p];
          bad |= id < 0 || id >= P.num_pages;
        }
      }
      if (tid == 0) sh.badv = 0;
      bad = soft_sync_or(bad);
      shift = -INFINITY;
      sum = 0.0f;
      int up = mine ? node : -1;  // next ancestor to pass
      const int mysteps = w.two ? T : (T + 1 - wg) / 2;
      for (int i = 0; i < mysteps; ++i) {
        const int tile = w.two ? i : 2 * i + wg, j = w.j0 + tile;
        const bool tree = j < w.s.tt;
        const int first = tree ? (w.s.tt - 1 - j) * kTile : (j - w.s.tt) * kTile;
        const int valid = min(kTile, (tree ? min(w.s.n, SV_MAX_NODES) : w.s.len) - first);
        uint32_t see[4] = {0, 0, 0, 0};
        if (tree) {  // ancestors that lie in this tile
          while (up >= first) {
            const int e = up - first;
            if (e < kTile) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if ((e >> 5) == q) see[q] |= 1u << (e & 31);
            }
            const int p = __ldg(parents + up);
            if (p < -1 || p >= up) {
              bad = true;
              up = -1;
            } else {
              up = p;
            }
          }
        }
        // rows of the value tile that hold no key of this tile weigh nothing, but a weight of
        // zero does not silence what they may hold: they are cleared, and so are infinities and
        // NaN in the nodes' own values (added back at the end to the rows that see them)
        if ((tree || valid < kTile) && (!w.two || wg == 0)) {
          const int vpos = t0 + 2 * tile + 1, st = vpos % S::kStages;
          if (alive) alive = __all_sync(0xffffffffu, wait(sh, &sh.full[st], (vpos / S::kStages) & 1));
          if (alive) {
            char* vt = ring + st * S::kTileBytes;
            if (r >= valid) {
              for (int hf = 0; hf < S::kHalves; ++hf)
                for (int c = 0; c < 8; ++c)
                  *reinterpret_cast<uint4*>(vt + hf * (kTile * 128) + r * 128 + ((c ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            } else if (tree) {
              for (int hf = 0; hf < S::kHalves; ++hf)
                for (int c = 0; c < 8; ++c) {
                  uint32_t* at = reinterpret_cast<uint32_t*>(vt + hf * (kTile * 128) + r * 128 + ((c ^ (r & 7)) << 4));
                  const uint4 x = *reinterpret_cast<uint4*>(at);
                  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const bool lo = not_finite<kBf16>(xs[e]), hi = not_finite<kBf16>(xs[e] >> 16);
                    if (lo || hi) {
                      at[e] = xs[e] & (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
                      sh.badv = 1;
                    }
                  }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        if (alive) alive = __all_sync(0xffffffffu, wait(sh, &sh.sfull[wg], steps_done & 1));
        ++steps_done;
        if (alive && busy) {
          tc_fence_after();
          if (tree) {
            weigh(std::integral_constant<int, 2>(), i == 0, mine, valid, see);
          } else if (valid < kTile) {
            weigh(std::integral_constant<int, 1>(), i == 0, mine, valid, nullptr);
          } else {
            weigh(std::integral_constant<int, 0>(), i == 0, mine, valid, nullptr);
          }
          tc_fence_before();
        }
        mbar_arrive(&sh.pready[wg]);
      }
      // ---- the part's result
      if (alive && mysteps > 0) alive = __all_sync(0xffffffffu, wait(sh, &sh.pvdone[wg], (steps_done - 1) & 1));
      if (bad || !alive) sum = NAN;
      sh.xch[wg][r] = make_float2(shift, sum);
      tc_fence_before();
      soft_sync();
      tc_fence_after();
      const bool join = !w.two;  // both groups hold parts of the same rows
      float f0 = 1.0f, f1 = 0.0f;
      if (join) {
        const float2 a = sh.xch[0][r], b = sh.xch[1][r];
        const float now = fmaxf(a.x, b.x);
        f0 = a.x == -INFINITY ? 0.0f : ex2_approx(a.x - now);
        f1 = b.x == -INFINITY ? 0.0f : ex2_approx(b.x - now);
        shift = now;
        sum = f0 * a.y + (T > 1 ? f1 * b.y : 0.0f);
      }
      const bool whole = w.j0 == 0 && w.j1 == w.s.J;
      const bool extra = sh.badv != 0;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int slot = cta * 2 + (dseg == 0 ? 0 : 1);
      const int row = w.s.lo + node;
      const int head = w.h * P.G + rg;
      const int cbeg = join ? wg * (DP / 2) : 0, cend = join ? cbeg + DP / 2 : DP;
      if (busy) {
#pragma unroll 1
        for (int c = cbeg; c < cend; c += 32) {
          float o[32];
          if (alive) {
            tmem_ld32(o_at + (join ? 0 : wg * kTile) + c, o);
            tc_wait_ld();
            if (join) {
              if (T > 1) {
                float o1[32];
                tmem_ld32(o_at + kTile + c, o1);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = f0 * o[e] + f1 * o1[e];
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = NAN;
          }
          if (extra && mine) {  // infinities and NaN among the values this row sees
            for (int a = node; a >= 0;) {
              const uint16_t* vr = P.v + (w.s.lo + a) * P.v_node + w.h * P.v_head;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c + e < P.D) {
                  const uint32_t x = __ldg(vr + c + e);
                  if (not_finite<kBf16>(x)) o[e] += widen<kBf16>(x);
                }
              const int p = __ldg(parents + a);
              a = p < a ? p : -1;
            }
          }
          if (mine) {
            if (whole) {
              uint16_t* out = static_cast<uint16_t*>(P.out) + (static_cast<int64_t>(row) * P.Hq + head) * P.D + c;
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                if (c + e < P.D)
                  *reinterpret_cast<uint4*>(out + e) =
                      make_uint4(pack2<kBf16>(o[e] * inv, o[e + 1] * inv), pack2<kBf16>(o[e + 2] * inv, o[e + 3] * inv),
                                 pack2<kBf16>(o[e + 4] * inv, o[e + 5] * inv), pack2<kBf16>(o[e + 6] * inv, o[e + 7] * inv));
            } else {
              float4* po = reinterpret_cast<float4*>(P.part_o) +
                           (static_cast<int64_t>(slot * 2 + (join ? 0 : wg)) * (DP / 4) + c / 4) * kTile + r;
#pragma unroll
              for (int e = 0; e < 32; e += 4) po[(e / 4) * kTile] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
      }
      if (mine && (!join || wg == 0)) {
        if (whole) {
          if (P.lse) P.lse[static_cast<int64_t>(row) * P.Hq + head] = (shift + log2f(sum)) * kLn2;
        } else {
          P.part_s[static_cast<int64_t>(slot * 2 + (join ? 0 : wg)) * kTile + r] = make_float2(shift, sum);
        }
      }
      // the unit starts here and goes on behind this CTA: describe it for the join
      if (tid == 0 && w.j0 == 0 && w.j1 < w.s.J) {
        P.desc[cta * 2] = make_int4(w.s.lo + w.u * 2 * P.npt, min(w.s.n - w.u * 2 * P.npt, 2 * P.npt), w.h, slot);
        P.desc[cta * 2 + 1] = make_int4(cdiv(w.s.J - w.j1, static_cast<int>(min(chunk, static_cast<int64_t>(INT_MAX)))), 0, 0, 0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.oempty);
      soft_sync();  // xch and badv are free again
      t0 += 2 * T;
      ++dseg;
    }
    if (tid == 0) {
      // no unit is cut behind this CTA
      const bool cut = dseg > 0 && w.j0 == 0 && w.j1 < w.s.J;
      if (!cut) P.desc[cta * 2] = make_int4(0, 0, 0, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Join of the units that CTA borders cut: block (x, y) takes 2^10 four-column
// groups of the unit that starts in CTA x and ends behind it.
template <int DP, bool kBf16>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x;
  const int4 d = P.desc[cta * 2];
  const int nodes = d.y;
  if (nodes == 0) return;
  const int more = P.desc[cta * 2 + 1].x;  // parts behind the first
  const int idx = blockIdx.y * 256 + threadIdx.x;
  const int r2 = idx % (2 * kTile), cg = idx / (2 * kTile);  // row of the two tiles, column group
  const int tile = r2 / kTile, r = r2 - tile * kTile;
  const int rnode = r / P.G, rg = r - rnode * P.G;
  if (rnode >= P.npt || tile * P.npt + rnode >= nodes || cg >= DP / 4) return;
  auto at = [&](int p) { return (p == 0 ? d.w : (cta + p) * 2) * 2 + tile; };
  float top = -INFINITY;
  for (int p = 0; p <= more; ++p) top = fmaxf(top, P.part_s[static_cast<int64_t>(at(p)) * kTile + r].x);
  float sum = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int p = 0; p <= more; ++p) {
    const float2 s = P.part_s[static_cast<int64_t>(at(p)) * kTile + r];
    const float4 x = reinterpret_cast<const float4*>(P.part_o)[(static_cast<int64_t>(at(p)) * (DP / 4) + cg) * kTile + r];
    const float f = s.x == -INFINITY ? 0.0f : ex2_approx(s.x - top);
    sum += f * s.y;
    o.x += f * x.x;
    o.y += f * x.y;
    o.z += f * x.z;
    o.w += f * x.w;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t row = static_cast<int64_t>(d.x + tile * P.npt + rnode) * P.Hq + d.z * P.G + rg;
  if (cg * 4 < P.D)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + row * P.D + cg * 4) =
        make_uint2(pack2<kBf16>(o.x * inv, o.y * inv), pack2<kBf16>(o.z * inv, o.w * inv));
  if (P.lse && cg == 0) P.lse[row] = (top + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static std::mutex mu;
  static EncodeFn fn;
  std::lock_guard<std::mutex> lk(mu);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  }
  return fn;
}

// A map over [.., D] with `rank` - 1 outer axes; the box is 64 elements by
// `box`.  An axis of size 1 takes any stride.
int make_map(EncodeFn enc, CUtensorMap* map, bool bf16, const void* base, int rank, const int64_t* size,
             const int64_t* stride, const int* box, const char* what) {
  cuuint64_t dims[5], strides[4];
  cuuint32_t boxes[5], ones[5];
  for (int i = 0; i < rank; ++i) {
    dims[i] = static_cast<cuuint64_t>(size[i]);
    boxes[i] = static_cast<cuuint32_t>(box[i]);
    ones[i] = 1;
    if (i > 0) strides[i - 1] = size[i] == 1 ? 16 : static_cast<cuuint64_t>(stride[i]) * 2;
  }
  const CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, boxes, ones,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(SV_ERR_INVALID_ARG, "%s: layout not accepted (driver status %d)", what, static_cast<int>(r));
  return SV_OK;
}

constexpr int kMaxCtas = 160;  // SMs of a device, with room

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct AttnLayout {
  size_t o, s, desc, total;
};
AttnLayout attn_layout(int D) {
  const int DP = D <= 64 ? 64 : 128;
  AttnLayout l{};
  size_t off = 0;
  l.o = off;
  off += up256(static_cast<size_t>(kMaxCtas) * 4 * kTile * DP * sizeof(float));
  l.s = off;
  off += up256(static_cast<size_t>(kMaxCtas) * 4 * kTile * sizeof(float2));
  l.desc = off;
  off += up256(static_cast<size_t>(kMaxCtas) * 2 * sizeof(int4));
  l.total = off;
  return l;
}

int sm_count(int* out) {
  static std::mutex mu;
  static int cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  std::lock_guard<std::mutex> lk(mu);
  int n = dev >= 0 && dev < 64 ? cached[dev] : 0;
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    if (dev >= 0 && dev < 64) cached[dev] = n;
  }
  *out = n < kMaxCtas ? n : kMaxCtas;
  return SV_OK;
}

template <int DP, bool kBf16>
int launch_attn(const AttnParams& p, int ctas, cudaStream_t stream) {
  constexpr size_t kSmem = Shape<DP>::kTiles + sizeof(Shared);
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<DP, kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmem));
  if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  attn_kernel<DP, kBf16><<<ctas, kThreads, kSmem, stream>>>(p);
  int rc = check_launch("tree attention");
  if (rc != SV_OK) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, DP / 4 * 2 * kTile / 256);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, combine_kernel<DP, kBf16>, p);
  if (e != cudaSuccess) return set_error(SV_ERR_CUDA, "tree attention join launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_tree_attention_workspace_size(int Hq, int Hkv, int D) {
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > kTile || D < 8 || D > SV_MAX_HEAD_DIM || D % 8) return 0;
  return attn_layout(D).total;
}

int spec_tree_attention(const sv_tree_attention_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a) return set_error(SV_ERR_INVALID_ARG, "args is NULL");
  if (a->dtype != SV_BF16 && a->dtype != SV_F16) return set_error(SV_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
  if (a->B < 0 || a->B > SV_MAX_BATCH)
    return set_error(SV_ERR_INVALID_ARG, "B must be in [0, %d] (got %d)", SV_MAX_BATCH, a->B);
  if (a->N < 0) return set_error(SV_ERR_INVALID_ARG, "N must be >= 0 (got %d)", a->N);
  if (a->Hkv < 1 || a->Hq < a->Hkv || a->Hq % a->Hkv || a->Hq / a->Hkv > kTile)
    return set_error(SV_ERR_INVALID_ARG, "Hq must be a multiple of Hkv, up to %d times (got %d, %d)", kTile, a->Hq, a->Hkv);
  if (a->D < 8 || a->D > SV_MAX_HEAD_DIM || a->D % 8)
    return set_error(SV_ERR_UNSUPPORTED, "D must be a multiple of 8 in [8, %d] (got %d)", SV_MAX_HEAD_DIM, a->D);
  const int pg = a->page_size;
  if (!(pg == 8 || pg == 16 || pg == 32 || pg == 64 || (pg >= 128 && pg % 128 == 0)))
    return set_error(SV_ERR_UNSUPPORTED, "page_size must be 8, 16, 32, 64 or a multiple of 128 (got %d)", pg);
  if (a->num_pages < 1 || a->table_width < 0)
    return set_error(SV_ERR_INVALID_ARG, "num_pages must be >= 1 and table_width >= 0 (got %d, %d)", a->num_pages, a->table_width);
  if (static_cast<int64_t>(a->table_width) * pg > INT_MAX - kTile)
    return set_error(SV_ERR_INVALID_ARG, "a table row of %d pages is too long", a->table_width);
  if (!(a->scale > 0.0f && a->scale < INFINITY))
    return set_error(SV_ERR_INVALID_ARG, "scale must be positive and finite");
  if (a->B == 0 || a->N == 0) return SV_OK;
  if (!a->q || !a->k || !a->v || !a->k_cache || !a->v_cache || !a->out || !a->lens || !a->parents || !a->cu_nodes ||
      (a->table_width > 0 && !a->block_table))
    return set_error(SV_ERR_INVALID_ARG, "NULL input or output pointer");
  if (misaligned(a->q, 16) || misaligned(a->k, 16) || misaligned(a->v, 16) || misaligned(a->k_cache, 16) ||
      misaligned(a->v_cache, 16) || misaligned(a->out, 16))
    return set_error(SV_ERR_INVALID_ARG, "q, k, v, the caches and out must be 16-byte aligned");
  if (misaligned(a->lens, 4) || misaligned(a->parents, 4) || misaligned(a->cu_nodes, 4) ||
      misaligned(a->block_table, 4) || misaligned(a->out_lse, 4))
    return set_error(SV_ERR_INVALID_ARG, "pointers must be aligned to their element size");
  struct {
    int64_t stride;
    int size;
  } axes[] = {{a->q_node, a->N}, {a->q_head, a->Hq}, {a->k_node, a->N}, {a->k_head, a->Hkv}, {a->v_node, a->N},
              {a->v_head, a->Hkv}, {a->kc_page, a->num_pages}, {a->kc_token, pg}, {a->kc_head, a->Hkv},
              {a->vc_page, a->num_pages}, {a->vc_token, pg}, {a->vc_head, a->Hkv}};
  for (const auto& x : axes)
    if (x.size > 1 && (x.stride < 8 || x.stride % 8))
      return set_error(SV_ERR_INVALID_ARG, "strides must be positive multiples of 8 elements (got %lld)",
                       static_cast<long long>(x.stride));
  const AttnLayout lay = attn_layout(a->D);
  if (!workspace || misaligned(workspace, 256))
    return set_error(SV_ERR_WORKSPACE, "workspace must be given and 256-byte aligned");
  if (workspace_bytes < lay.total)
    return set_error(SV_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes, lay.total);
  int rc = check_device();
  if (rc != SV_OK) return rc;
  int ctas = 0;
  if ((rc = sm_count(&ctas)) != SV_OK) return rc;
  const EncodeFn enc = encoder();
  if (!enc) return set_error(SV_ERR_CUDA, "the driver offers no cuTensorMapEncodeTiled");

  AttnParams p{};
  const bool bf16 = a->dtype == SV_BF16;
  const int G = a->Hq / a->Hkv, npt = kTile / G, box = pg < kTile ? pg : kTile;
  {
    const int64_t qs[3] = {a->D, a->Hq, a->N}, qst[3] = {1, a->q_head, a->q_node};
    const int qb[3] = {64, G, npt};
    const int64_t ks[3] = {a->D, a->Hkv, a->N};
    const int64_t kst[3] = {1, a->k_head, a->k_node}, vst[3] = {1, a->v_head, a->v_node};
    const int kb[3] = {64, 1, kTreeBox};
    const int64_t cs[4] = {a->D, pg, a->Hkv, a->num_pages};
    const int64_t kcst[4] = {1, a->kc_token, a->kc_head, a->kc_page}, vcst[4] = {1, a->vc_token, a->vc_head, a->vc_page};
    const int cb[4] = {64, box, 1, 1};
    if ((rc = make_map(enc, &p.qmap, bf16, a->q, 3, qs, qst, qb, "q")) != SV_OK ||
        (rc = make_map(enc, &p.kmap, bf16, a->k, 3, ks, kst, kb, "k")) != SV_OK ||
        (rc = make_map(enc, &p.vmap, bf16, a->v, 3, ks, vst, kb, "v")) != SV_OK ||
        (rc = make_map(enc, &p.kcmap, bf16, a->k_cache, 4, cs, kcst, cb, "k_cache")) != SV_OK ||
        (rc = make_map(enc, &p.vcmap, bf16, a->v_cache, 4, cs, vcst, cb, "v_cache")) != SV_OK)
      return rc;
  }
  p.out = a->out;
  p.lse = a->out_lse;
  p.table = a->block_table;
  p.lens = a->lens;
  p.parents = a->parents;
  p.cu = a->cu_nodes;
  p.v = static_cast<const uint16_t*>(a->v);
  p.v_node = a->v_node;
  p.v_head = a->v_head;
  p.table_row = a->table_row;
  p.B = a->B;
  p.N = a->N;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = G;
  p.D = a->D;
  p.num_pages = a->num_pages;
  p.page = pg;
  p.width = a->table_width;
  p.box = box;
  p.npt = npt;
  p.sl = a->scale * kLog2e;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws + lay.o);
  p.part_s = reinterpret_cast<float2*>(ws + lay.s);
  p.desc = reinterpret_cast<int4*>(ws + lay.desc);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->D <= 64) return bf16 ? launch_attn<64, true>(p, ctas, s) : launch_attn<64, false>(p, ctas, s);
  return bf16 ? launch_attn<128, true>(p, ctas, s) : launch_attn<128, false>(p, ctas, s);
}

}  // extern "C"

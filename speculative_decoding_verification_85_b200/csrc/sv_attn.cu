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
// One CTA: four warps fill a ring of key and value tiles by TMA; two groups of
// four softmax warps turn scores S = Q K^T (fp32, tensor memory) into weights P
// (a thread a row: maximum, exponentials and sum need no exchange), each fed by
// one warp that issues its S and one that issues its O += P V.  With two query
// tiles both groups take every key tile; with one the groups take the key tiles
// in turn and their results are joined at the end (each reads the other's
// accumulator: same lanes).  A step is 64 keys, and a group has two score
// buffers: while it weighs one step, the next step's scores are made and the
// last one's weights used.  The accumulator is rescaled only when a row's
// maximum has grown by more than 2^8; until then weights up to 2^8 (fp16: 2^15,
// see kHold) are accumulated, which fp32 holds as well.
//
// Bound by memory while a key head has one tile of query rows.  Measured (1.08 GB
// of keys and values, 64 x 4096 tokens, 8 key heads of 128, pages of 128): 182 us
// with 4 rows a key head (0.90 of the measured copy bandwidth), 188 with 20, 210
// with 128 (0.79), 335 with 256 (two groups of 128 exponentials a key each):
// there the chain scores -> weights -> accumulator -> next scores of a group sets
// the pace, and products and exponentials take turns, at half of the tensor pipe
// and of the special function units.  Pages of 16 take the same 188 us with 20
// rows.  Contexts of 1 to 8192 tokens with as many bytes take 203: the line is
// cut by a count of tiles, in which a partial tile stands for a whole one and the
// start and end of a unit for nothing.
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
constexpr int kHalf = 64;           // keys of a step
constexpr int kWarpsSoft = 8;       // softmax warps: two groups of four
// Warps 0-7: softmax; 8: keys, 9: values; 10 and 11: first products of each
// softmax group; 12 and 13: second products (apart, since each would wait for
// the other's turn); 14 and 15: keys and values beyond the first 64 columns of
// a head (small pages are many loads).
constexpr int kWarpK = 8, kWarpS = 10, kWarpO = 12, kWarpMore = 14;
constexpr int kThreads = 32 * 16;
// Registers: the softmax groups hold 64 scores a thread, the others need few.
// 2 x 168 + 2 x 88 = 4 x 128, what a block of 512 threads is launched with.
constexpr int kRegsSoft = 168, kRegsRest = 88;
constexpr float kGrow = 8.0f;       // base-2 growth of a maximum that is let stand
// A row's exponent shift lies this far below its maximum (base 2).  In fp16 weights below 2^-14
// lose bits and those below 2^-25 vanish; carried 2^7 higher, the largest stays below
// 2^(7 + kGrow) and one that is 2^-21 of it is still rounded by 2^-11 of itself.  (11 with a
// growth of 4 costs 2% on 16 trees of 64 nodes, 440 us against 432; 7 with 8 costs nothing.)
// bf16 has fp32's exponents and needs none.
template <bool kBf16>
constexpr float kHold = kBf16 ? 0.0f : 7.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCtas = 160;         // SMs of a device, with room
constexpr int kTreeBox = 16;        // rows of one load of the nodes' own keys and values

// Ring of key and value tiles.  Tile t of the CTA goes to pair t % kPairs: its
// keys to stage 2 (t % kPairs), its values to the next one, lap t / kPairs.
// With one query tile group t % 2 takes tile t, with two query tiles both do.
// The number of pairs is even, so in either mode a group passes every lap of
// the pairs of its own parity; it passes all laps of the others once both
// groups have met at the start of a part with two query tiles.  A barrier's
// parity therefore never stands for a lap that a waiter has not seen.
template <int DP>
struct Shape {
  static constexpr int kHalves = DP / 64;
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kPairs = DP == 128 ? 2 : 4;
  static constexpr size_t kTiles = static_cast<size_t>(2 + 2 * kPairs) * kTileBytes;
  static __device__ __forceinline__ int stage(int t) { return 2 * (t % kPairs); }
  static __device__ __forceinline__ uint32_t parity(int t) { return (t / kPairs) & 1; }
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
  int ctas, groups;    // CTAs; column groups of four of a partial result
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
  const int lo = P.cu[b], hi = P.cu[b + 1], len = P.lens[b];
  Seq s{};
  if (lo < 0 || hi > P.N || hi <= lo) return s;
  s.lo = lo;
  s.n = hi - lo;
  s.mark = s.n > SV_MAX_NODES || len < 0 || len > static_cast<int64_t>(P.width) * P.page;
  s.len = s.mark ? 0 : len;
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

// One part as the other warps read it: the key warp walks the line and leaves
// every part's description in a ring of kParts.
struct alignas(16) Part {
  int lo, n, len, tt;     // first packed row, nodes, cached tokens, tree tiles
  int h, u, j0, j1;       // key head, unit within the head, tiles of the unit
  int J, b, two, mark;    // tiles of the whole unit, sequence; two query tiles; marked; b < 0: the end
};
constexpr int kParts = 8;

struct Shared {
  uint64_t full[8], empty[8];
  uint64_t sfull[2][2], pready[2][2], pvdone[2][2];  // [group][step & 1]
  uint64_t qfull[2], oempty[2], drain[4], meet[2], met;
  float2 xch[2][kTile];       // [group][row]: shift, sum
  int64_t scan[16];
  Walk start;                 // the stretch (left == 0: nothing for this CTA)
  int64_t chunk;              // tiles of a stretch
  uint32_t tmem;
  int dead;
  int badv[4];                // [part & 3]: a tree tile holds infinities or NaN among its values
  int badpage[kParts];        // a page outside the cache
  uint64_t parted[kParts], freed[kParts];  // the part is described; all readers are done with it
  Part parts[kParts];
};

// Wait for a phase; false once any wait of the CTA has run out of time.  (Kept
// short: it is inlined at every wait, and instruction fetches are part of what
// this kernel waits for.)
__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  volatile int* dead = &sh.dead;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*dead) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *dead = 1;
      return false;
    }
  }
  return true;
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
__device__ __forceinline__ bool any_not_finite(const uint4& y) {
  constexpr uint32_t m = kExpMask<kBf16> * 0x10001u;
  return (__vcmpeq2(y.x & m, m) | __vcmpeq2(y.y & m, m) | __vcmpeq2(y.z & m, m) | __vcmpeq2(y.w & m, m)) != 0;
}
template <bool kBf16>
__device__ __forceinline__ float widen(uint32_t half) {
  if constexpr (kBf16) return __uint_as_float(half << 16);
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<uint16_t>(half)));
  return f;
}

// A row sees itself at least; its sum is zero only where every score it sees is -inf, and its
// output is 0 / 0 then, whatever the accumulator holds.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? NAN : 1.0f / sum; }

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
    for (int i = 0; i < 2 * S::kPairs; ++i) {
      mbar_init(&sh.full[i], S::kHalves);  // a loading warp for each 64 columns
      mbar_init(&sh.empty[i], 2);  // both groups' products
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qfull[i], 1);
      for (int e = 0; e < 2; ++e) {
        mbar_init(&sh.sfull[i][e], 1);
        mbar_init(&sh.pready[i][e], kTile);
        mbar_init(&sh.pvdone[i][e], 1);
      }
      mbar_init(&sh.oempty[i], kWarpsSoft);
      mbar_init(&sh.meet[i], 2);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.drain[i], 1);
    mbar_init(&sh.met, kWarpsSoft);
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&sh.parted[i], 1);
      mbar_init(&sh.freed[i], kWarpsSoft + 2 * S::kHalves - 1 + 4);  // softmax, loads but the first, products
    }
    for (int i = 0; i < 4; ++i) sh.badv[i] = 0;
    mbar_init_fence();
    sh.dead = 0;
  }
  if (tid >= 32 && tid < 37) {  // the maps, while the stretch is worked out
    const CUtensorMap* maps = &P.qmap;
    asm volatile("prefetch.tensormap [%0];" ::"l"(maps + (tid - 32)) : "memory");
  }
  if (warp == kWarpS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();

  // ---- where this CTA's stretch begins: prefix sums of the sequences' tiles.  The key warp
  // alone walks the line; for a few sequences it also finds the start alone, while the others
  // set up, else the whole block does.  (One node and 100 tokens a sequence, key warp / block:
  // 1 sequence 10.7 / 11.4 us, 16: 11.9 / 12.6, 64: 12.5 / 12.3, 128: 18.2 / 16.1, 256: 32 / 26.)
  const bool few = P.B <= 128;
  auto find_start = [&](auto wide) {
    constexpr bool kWide = decltype(wide)::value;
    constexpr int kLanes = kWide ? kThreads : 32;
    const int me = kWide ? tid : lane;
    int64_t total = 0, chunk = 0, begin = 0;
    if (me == 0) sh.start.left = 0;
    __syncwarp();
    for (int pass = 0; pass < 2; ++pass) {  // the total, then the sequence that `begin` lies in
      int64_t carry = 0;
#pragma unroll 1
      for (int base = 0; base < P.B; base += kLanes) {
        const int b = base + me;
        Seq s{};
        if (b < P.B) s = seq_of(P, b);
        const int64_t mine = static_cast<int64_t>(s.J) * s.U * P.Hkv;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int64_t sum = __shfl_sync(0xffffffffu, incl, 31);
        if constexpr (kWide) {
          __syncthreads();
          if (lane == 31) sh.scan[warp] = incl;
          __syncthreads();
          sum = 0;
          for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) incl += sh.scan[i];
            sum += sh.scan[i];
          }
        }
        incl += carry;
        carry += sum;
        if (pass == 1 && mine > 0 && incl - mine <= begin && begin < incl) {
          Walk k{};
          const int64_t at = begin - (incl - mine);
          k.b = b;
          k.s = s;
          k.hu = static_cast<int>(at / s.J);
          k.j = static_cast<int>(at - static_cast<int64_t>(k.hu) * s.J);
          k.left = min(chunk, total - begin);
          sh.start = k;
        }
      }
      if (pass == 0) {
        total = carry;
        chunk = (total + gridDim.x - 1) / gridDim.x;
        begin = cta * chunk;
      }
    }
    if (me == 0) sh.chunk = chunk;
  };
  if (!few) find_start(std::true_type());
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // Part `seg`; every reader takes them all, in order, and gives each back (freed).
  // Keys of tile j of a unit; a tile of more than kHalf takes two steps.
  auto keys_of = [&](const Part& w, int j) {
    return min(kTile, j < w.tt ? min(w.n, SV_MAX_NODES) - (w.tt - 1 - j) * kTile : w.len - (j - w.tt) * kTile);
  };
  auto part_of = [&](int seg, Part& w) {
    const bool ok = wait(sh, &sh.parted[seg % kParts], (seg / kParts) & 1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const int4* d = reinterpret_cast<const int4*>(&sh.parts[seg % kParts]);
    int4* o = reinterpret_cast<int4*>(&w);
    o[0] = d[0];
    o[1] = d[1];
    o[2] = d[2];
    // one lane gives the place back for the whole warp: not before every lane has read it
    __syncwarp();
    return w.b >= 0;
  };

  if (warp >= kWarpsSoft) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp < kWarpS || (S::kHalves == 2 && warp >= kWarpMore)) {
      // -------------------------------------------------- keys and values
      // a warp for each and for each 64 columns of a head; the first one also walks the line
      const bool kv = warp & 1, lead = warp == kWarpK;
      const int hf = warp >= kWarpMore;
      const CUtensorMap* own = kv ? &P.vmap : &P.kmap;
      const CUtensorMap* cached = kv ? &P.vcmap : &P.kcmap;
      int t = 0, seg = 0;
      bool ok = true;
      Walk walk{};
      if (lead) {
        if (few) find_start(std::false_type());
        __syncwarp();
        walk = sh.start;
      }
      for (;; ++seg) {
        Part w;
        if (!lead) {
          if (!part_of(seg, w)) break;
          if (lane == 0) mbar_arrive(&sh.freed[seg % kParts]);
        } else {
          w.b = -1;
          ok = ok && __all_sync(0xffffffffu, wait(sh, &sh.freed[seg % kParts], ((seg / kParts) & 1) ^ 1));
          if (!ok) break;
          if (walk.next(P))
            w = {walk.s.lo, walk.s.n, walk.s.len, walk.s.tt, walk.h, walk.u, walk.j0, walk.j1, walk.s.J, walk.b, walk.two, walk.s.mark};
          if (lane == 0) {
            sh.badpage[seg % kParts] = 0;
            sh.parts[seg % kParts] = w;
            mbar_arrive(&sh.parted[seg % kParts]);
          }
          __syncwarp();
          if (w.b < 0) break;
          // the parents' lines, which the softmax warps will walk
          if (w.j0 < w.tt && lane * 32 < w.n)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(P.parents + w.lo + lane * 32));
        }
        const int32_t* row = P.table + w.b * P.table_row;
        // this lane's page of a context tile (read a tile ahead): its load's page where pages
        // are smaller than a tile, else the tile's
        const int per = kTile / P.box, span = P.page / P.box;
        auto page_at = [&](int j) {
          const int c = j - w.tt;
          if (c < 0 || j >= w.j1 || lane >= per || c * kTile + lane * P.box >= w.len) return 0;
          return row[span == 1 ? c * per + lane : c / span];
        };
        int page = page_at(w.j0);
        for (int j = w.j0; j < w.j1; ++j) {
          const int ahead = page_at(j + 1);
          const bool tree = j < w.tt;
          const int c = tree ? w.tt - 1 - j : j - w.tt;  // tile of the tree, of the context
          const int valid = min(kTile, (tree ? min(w.n, SV_MAX_NODES) : w.len) - c * kTile);
          const int rows = tree ? kTreeBox : P.box;
          const int boxes = (valid + rows - 1) / rows;
          if (page < 0 || page >= P.num_pages) {
            if (lead) sh.badpage[seg % kParts] = 1;  // the rows will be marked
            page = 0;
          }
          const int st = S::stage(t) + (kv ? 1 : 0);
          ok = __all_sync(0xffffffffu, wait(sh, &sh.empty[st], S::parity(t) ^ 1));
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], boxes * rows * 128);
          __syncwarp();
          if (lane < boxes) {
            char* dst = ring + st * S::kTileBytes + hf * (kTile * 128) + lane * rows * 128;
            if (tree) {
              tma_3d(dst, own, hf * 64, w.h, w.lo + c * kTile + lane * kTreeBox, &sh.full[st]);
            } else {
              const int tok = span == 1 ? 0 : (c % span) * kTile;
              tma_4d(dst, cached, hf * 64, tok, w.h, page, &sh.full[st]);
            }
          }
          __syncwarp();
          page = ahead;
          ++t;
        }
        if (!ok) break;
      }
      // leave no copy in flight behind (the others may have given up)
      for (int i = max(0, t - S::kPairs); i < t; ++i) {
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(&sh.full[S::stage(i) + (kv ? 1 : 0)], S::parity(i)) && global_ns() - t0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    } else if (warp < kWarpMore) {
      // --------------------------------------------------------- products
      // a warp for each kind and softmax group; the whole warp keeps the books, one lane issues
      const int s = (warp - kWarpS) & 1;
      const bool issuer = elect_one();
      constexpr int kStep = S::kTileBytes >> 4;       // from one tile's descriptor to the next's
      constexpr int kHalfStep = (kHalf * 128) >> 4;   // from a tile's first keys to its second ones
      const uint32_t s_at = tmem + s * kTile, o_at = tmem + 2 * kTile + s * kTile;
      int t0 = 0, seg = 0;              // tiles and parts so far
      uint32_t n = 0, ntwo = 0;         // products, parts with two query tiles so far
      bool ok = true;
      Part w;
      auto next_part = [&]() {
        const bool got = part_of(seg, w);
        if (issuer && got) mbar_arrive(&sh.freed[seg % kParts]);
        ++seg;
        return got;
      };
      // this group's tiles in the part that begins at tile t
      auto tiles_of = [&]() {
        const int T = w.j1 - w.j0;
        return w.two ? T : (T + 1 - ((s ^ t0) & 1)) / 2;
      };
      // before a part with two query tiles: the other group has passed all tiles up to here, too
      auto meet = [&](uint64_t* bar) {
        if (issuer) mbar_arrive(bar);
        return __all_sync(0xffffffffu, wait(sh, bar, ntwo++ & 1));
      };
      bool more = next_part();
      if (warp < kWarpO) {
        // S of a step's keys, step n into buffer n % 2 once its weights of two steps ago are used
        constexpr uint32_t idesc = instr_desc(kBf16, kHalf, false);
        const int ksteps = cdiv(P.D, 16);
        const uint64_t qdesc = smem_desc(smem_addr(qtile) + s * S::kTileBytes, 16);
        const uint64_t kdesc = smem_desc(smem_addr(ring), 16);
        uint32_t nq = 0;  // query tiles so far: the group's own copy
        while (ok && more) {
          const bool two = w.two;
          const int tiles = tiles_of(), stride = two ? 1 : 2;
          int t = two ? t0 : t0 + ((s ^ t0) & 1), j = w.j0 + t - t0;
          if (tiles > 0) {
            // the query tile's place is free once the last S from it is complete
            if (n > 0) ok = __all_sync(0xffffffffu, wait(sh, &sh.sfull[s][(n - 1) & 1], ((n - 1) >> 1) & 1));
            if (!ok) break;
            if (issuer) {
              mbar_arrive_expect_tx(&sh.qfull[s], P.npt * P.G * 128 * S::kHalves);
#pragma unroll
              for (int hf = 0; hf < S::kHalves; ++hf)
                tma_3d(qtile + s * S::kTileBytes + hf * (kTile * 128), &P.qmap, hf * 64, w.h * P.G,
                       w.lo + (w.u * 2 + (two ? s : 0)) * P.npt, &sh.qfull[s]);
            }
            __syncwarp();
            ++nq;
          }
          if (two) ok = meet(&sh.meet[0]);
          if (ok && tiles > 0) ok = __all_sync(0xffffffffu, wait(sh, &sh.qfull[s], (nq - 1) & 1));
          for (int i = 0; ok && i < tiles; ++i, t += stride, j += stride) {
            const int st = S::stage(t), halves = keys_of(w, j) > kHalf ? 2 : 1;
            ok = __all_sync(0xffffffffu, wait(sh, &sh.full[st], S::parity(t)));
            for (int h = 0; ok && h < halves; ++h) {
              const int buf = n & 1;
              ok = n < 2 || __all_sync(0xffffffffu, wait(sh, &sh.pvdone[s][buf], ((n >> 1) - 1) & 1));
              if (!ok) break;
              tc_fence_after();
              if (issuer) {
                const uint64_t db = kdesc + st * kStep + h * kHalfStep;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                  const int off = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;
                  if (k < ksteps) mma_ss(s_at + buf * kHalf, qdesc + off, db + off, idesc, k > 0);
                }
                mma_commit(&sh.sfull[s][buf]);
                if (h == halves - 1) {
                  mma_commit(&sh.empty[st]);
                  if (!two) mma_commit(&sh.empty[st]);  // (the other group's share)
                }
              }
              __syncwarp();
              ++n;
            }
          }
          t0 += w.j1 - w.j0;
          more = ok && next_part();
        }
        const uint64_t ts = global_ns();  // the copy in flight, if any
        while (nq > 0 && !mbar_try_wait(&sh.qfull[s], (nq - 1) & 1) && global_ns() - ts < kWaitLimitNs) {
        }
      } else {
        // O += P V
        constexpr uint32_t idesc = instr_desc(kBf16, DP, true);
        const uint64_t vdesc = smem_desc(smem_addr(ring), kTile * 128);
        uint32_t nown = 0;  // parts with tiles of this group so far
        while (ok && more) {
          const bool two = w.two;
          const int tiles = tiles_of(), stride = two ? 1 : 2;
          int t = two ? t0 : t0 + ((s ^ t0) & 1), j = w.j0 + t - t0;
          if (two) ok = meet(&sh.meet[1]);
          if (ok && tiles > 0 && nown++ > 0) ok = __all_sync(0xffffffffu, wait(sh, &sh.oempty[s], (nown - 2) & 1));
          for (int i = 0; ok && i < tiles; ++i, t += stride, j += stride) {
            const int st = S::stage(t) + 1, halves = keys_of(w, j) > kHalf ? 2 : 1;
            ok = __all_sync(0xffffffffu, wait(sh, &sh.full[st], S::parity(t)));
            for (int h = 0; ok && h < halves; ++h) {
              const int buf = n & 1;
              ok = __all_sync(0xffffffffu, wait(sh, &sh.pready[s][buf], (n >> 1) & 1));
              if (!ok) break;
              tc_fence_after();
              if (issuer) {
                const uint64_t db = vdesc + st * kStep + h * kHalfStep;
#pragma unroll
                for (int q = 0; q < kHalf / 16; ++q)
                  mma_ts(o_at, s_at + buf * kHalf + q * 8, db + q * (2048 >> 4), idesc, q > 0 || h > 0 || i > 0);
                mma_commit(&sh.pvdone[s][buf]);
                if (h == halves - 1) {
                  mma_commit(&sh.empty[st]);
                  if (!two) mma_commit(&sh.empty[st]);
                }
              }
              __syncwarp();
              ++n;
            }
          }
          t0 += w.j1 - w.j0;
          more = ok && next_part();
        }
      }
      // the products in flight
      if (issuer) mma_commit(&sh.drain[warp - kWarpS]);
      const uint64_t ts = global_ns();
      while (!mbar_try_wait(&sh.drain[warp - kWarpS], 0) && global_ns() - ts < kWaitLimitNs) {
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
    int t0 = 0, dseg = 0;       // tiles and parts so far
    uint32_t step = 0;          // steps of this group so far
    bool alive = true;
    float shift = 0.0f, sum = 0.0f;  // this row's exponent shift (base 2) and sum of weights

    // S of one step's keys to P: shift, sum and, when a maximum has grown much, the accumulator
    // (once the second product of the step before is done).  False: a wait failed.
    auto weigh = [&](bool fresh, bool mine) {
      const uint32_t at = s_at + (step & 1) * kHalf;
      float x[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) tmem_ld32(at + c, x + c);
      tc_wait_ld();
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < kHalf; c += 2) mx[(c >> 1) & 3] = fmaxf(fmaxf(mx[(c >> 1) & 3], x[c]), x[c + 1]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl - kHold<kBf16>;  // the shift it asks for
      if (fresh) {
        shift = top;
      } else if (__any_sync(0xffffffffu, mine && top - shift > kGrow)) {
        if (!__all_sync(0xffffffffu, wait(sh, &sh.pvdone[wg][(step - 1) & 1], ((step - 1) >> 1) & 1))) return false;
        tc_fence_after();
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
      for (int c0 = 0; c0 < kHalf; c0 += 32) {
        // weights rounded to the input type, which the second product needs: by 2^-8 (bf16) or
        // 2^-11 (fp16) relative at most, as the output itself is, and averaged over the keys;
        // in fp16 by 2^-25 where that is more, 2^-32 of the row's largest or less (kHold).
        // The sum takes them unrounded.
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const uint64_t y = fma2(pair(x[c0 + c], x[c0 + c + 1]), sl2, neg2);
          const float a = ex2_approx(pair_lo(y)), b = ex2_approx(pair_hi(y));
          part[(c >> 1) & 1] = add2(part[(c >> 1) & 1], pair(a, b));
          pk[c >> 1] = pack2<kBf16>(a, b);
        }
        tmem_st16(at + (c0 >> 1), pk);
      }
      const uint64_t p = add2(part[0], part[1]);
      sum += pair_lo(p) + pair_hi(p);
      tc_wait_st();
      return true;
    };

    Part w;
    bool cut = false;  // the last part's unit starts here and goes on behind this CTA
    int4 cut_at = make_int4(0, 0, 0, 0);
    int cut_left = 0;
    while (alive && part_of(dseg, w)) {
      const int T = w.j1 - w.j0, buf = dseg & 3;
      const int node = w.u * 2 * P.npt + (w.two ? wg * P.npt : 0) + rnode;  // within the sequence
      const bool mine = rnode < P.npt && node < w.n;
      const bool busy = __any_sync(0xffffffffu, mine);  // does this warp hold a row at all
      const int32_t* parents = P.parents + w.lo;
      bool bad = w.mark;
      shift = -INFINITY;
      sum = 0.0f;
      int up = mine ? node : -1;  // next ancestor to pass
      // the groups' tiles in this part (with one query tile tile t is group t % 2's)
      const int tiles0 = w.two ? T : (T + 1 - (t0 & 1)) / 2, tiles1 = w.two ? T : T - tiles0;
      const int mytiles = wg ? tiles1 : tiles0;
      for (int i = 0; alive && i < mytiles; ++i) {
        const int tile = w.two ? i : 2 * i + ((wg ^ t0) & 1), j = w.j0 + tile;
        const bool tree = j < w.tt;
        const int first = (tree ? w.tt - 1 - j : j - w.tt) * kTile;
        const int valid = keys_of(w, j);
        const bool special = tree || valid < kTile;
        uint32_t see[4];
        if (special) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int m = valid - 32 * q;
            see[q] = tree || m <= 0 ? 0u : (m >= 32 ? 0xFFFFFFFFu : (1u << m) - 1u);
          }
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
        }
#pragma unroll 1
        for (int half = 0; half * kHalf < valid; ++half) {
          alive = __all_sync(0xffffffffu, wait(sh, &sh.sfull[wg][step & 1], (step >> 1) & 1));
          if (!alive) break;
          if (busy) {
            tc_fence_after();
            if (special) {  // -inf for the keys that do not count
              const uint32_t at = s_at + (step & 1) * kHalf;
#pragma unroll 1
              for (int q = 0; q < 2; ++q) {
                const uint32_t m = half ? (q ? see[3] : see[2]) : (q ? see[1] : see[0]);
                float x[32];
                tmem_ld32(at + 32 * q, x);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(m >> c & 1)) x[c] = -INFINITY;
                tmem_st32(at + 32 * q, reinterpret_cast<uint32_t*>(x));
              }
              tc_wait_st();
            }
            alive = weigh(i == 0 && half == 0, mine);
            if (!alive) break;
            tc_fence_before();
          }
          if (special && half == 0) {
            // Rows of the value tile that hold no key of this tile weigh nothing, but a weight of
            // zero does not silence what they may hold: they are cleared, and so are infinities
            // and NaN in the nodes' own values (added back at the end to the rows that see them).
            // With two query tiles both groups do it, to the same effect.  (S of this tile says
            // that the second product two steps ago is done, and a tile of one step only is
            // special itself: the last lap of the value stage has been seen to be over.)
            const int st = S::stage(t0 + tile) + 1;
            alive = __all_sync(0xffffffffu, wait(sh, &sh.full[st], S::parity(t0 + tile)));
            if (!alive) break;
            char* vt = ring + st * S::kTileBytes + r * 128;
            if (r >= valid) {
#pragma unroll
              for (int c = 0; c < 8 * S::kHalves; ++c)
                *reinterpret_cast<uint4*>(vt + (c >> 3) * (kTile * 128) + (((c ^ r) & 7) << 4)) = make_uint4(0, 0, 0, 0);
            } else if (tree) {
              bool hit = false;
#pragma unroll
              for (int c = 0; c < 8 * S::kHalves; ++c) {
                const uint4 y = *reinterpret_cast<const uint4*>(vt + (c >> 3) * (kTile * 128) + (((c ^ r) & 7) << 4));
                hit |= any_not_finite<kBf16>(y);
              }
              if (hit) {
                sh.badv[buf] = 1;
                for (int c = 0; c < 64 * S::kHalves; ++c) {
                  uint16_t* v = reinterpret_cast<uint16_t*>(vt + (c >> 6) * (kTile * 128)) + (c & 63);
                  if (not_finite<kBf16>(*v)) *v = 0;
                }
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          mbar_arrive(&sh.pready[wg][step & 1]);
          ++step;
        }
      }
      if (!alive) break;
      // ---- the part's result
      if (mytiles > 0) alive = __all_sync(0xffffffffu, wait(sh, &sh.pvdone[wg][(step - 1) & 1], ((step - 1) >> 1) & 1));
      if (!alive) break;
      if (bad) sum = NAN;
      // (A group writes here again behind second products that wait for all warps to have left
      // its last part with steps; badv of two parts ahead was last read two meetings ago.)
      if (mytiles > 0) sh.xch[wg][r] = make_float2(shift, sum);
      if (tid == 0) sh.badv[(buf + 2) & 3] = 0;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.met);
      alive = __all_sync(0xffffffffu, wait(sh, &sh.met, dseg & 1));
      if (!alive) break;
      tc_fence_after();
      const bool extra = sh.badv[buf] != 0;
      const bool join = !w.two;  // both groups hold parts of the same rows
      float f0 = 1.0f, f1 = 0.0f;
      if (join) {
        const float2 a = tiles0 > 0 ? sh.xch[0][r] : make_float2(-INFINITY, 0.0f);
        const float2 b = tiles1 > 0 ? sh.xch[1][r] : make_float2(-INFINITY, 0.0f);
        const float now = fmaxf(a.x, b.x);
        f0 = a.x == -INFINITY ? 0.0f : ex2_approx(a.x - now);
        f1 = b.x == -INFINITY ? 0.0f : ex2_approx(b.x - now);
        shift = now;
        sum = f0 * a.y + f1 * b.y;
        if (bad) sum = NAN;
      }
      if (*const_cast<volatile int*>(&sh.badpage[dseg % kParts])) sum = NAN;
      const bool whole = w.j0 == 0 && w.j1 == w.J;
      const float inv = inverse(sum);
      const int slot = cta * 2 + (dseg == 0 ? 0 : 1);
      const int row = w.lo + node;
      const int head = w.h * P.G + rg;
      const int cbeg = join ? wg * (DP / 2) : 0, cend = join ? cbeg + DP / 2 : DP;
      if (busy) {
#pragma unroll 1
        for (int c = cbeg; c < cend; c += 16) {
          // with steps of one group alone, its accumulator is the result
          float o[16];
          tmem_ld16(o_at + (join ? tiles0 == 0 : wg) * kTile + c, o);
          if (join && T > 1) {
            float o1[16];
            tmem_ld16(o_at + kTile + c, o1);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = f0 * o[e] + f1 * o1[e];
          } else {
            tc_wait_ld();
          }
          if (extra && mine) {
            // infinities and NaN among the values this row sees in this part's tiles (one in
            // another part's tiles is added there: a part without a key of the row weighs
            // nothing in the join, and 0 * inf is NaN)
            const int from = max(w.tt - w.j1, 0) * kTile, to = (w.tt - w.j0) * kTile;
            for (int a = node; a >= from;) {
              const uint16_t* vr = P.v + (w.lo + a) * P.v_node + w.h * P.v_head;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (a < to && c + e < P.D) {
                  const uint32_t x = __ldg(vr + c + e);
                  if (not_finite<kBf16>(x)) o[e] += widen<kBf16>(x);
                }
              const int p = __ldg(parents + a);
              a = p < a ? p : -1;
            }
          }
          if (mine && c < P.D) {
            if (whole) {
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = pack2<kBf16>(o[2 * e] * inv, o[2 * e + 1] * inv);
              uint16_t* out = static_cast<uint16_t*>(P.out) + (static_cast<int64_t>(row) * P.Hq + head) * P.D + c;
              *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
              if (c + 8 < P.D) *reinterpret_cast<uint4*>(out + 8) = make_uint4(y[4], y[5], y[6], y[7]);
            } else {
              float4* po = reinterpret_cast<float4*>(P.part_o) +
                           (static_cast<int64_t>(slot * 2 + (join ? 0 : wg)) * (DP / 4) + c / 4) * kTile + r;
#pragma unroll
              for (int e = 0; e < 16; e += 4) po[(e / 4) * kTile] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (tiles0 > 0) mbar_arrive(&sh.oempty[0]);
        if (tiles1 > 0) mbar_arrive(&sh.oempty[1]);
      }
      if (mine && (!join || wg == 0)) {
        if (whole) {
          if (P.lse) P.lse[static_cast<int64_t>(row) * P.Hq + head] = (shift + log2f(sum)) * kLn2;
        } else {
          P.part_s[static_cast<int64_t>(slot * 2 + (join ? 0 : wg)) * kTile + r] = make_float2(shift, sum);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.freed[dseg % kParts]);
      t0 += T;
      ++dseg;
      cut = w.j0 == 0 && w.j1 < w.J;
      cut_at = make_int4(w.lo + w.u * 2 * P.npt, min(w.n - w.u * 2 * P.npt, 2 * P.npt), w.h, slot);
      cut_left = w.J - w.j1;
    }
    if (tid == 0) {
      // for the join: the cut unit's first node, nodes, key head, slot; parts behind this one
      const int more = cut ? static_cast<int>((cut_left + sh.chunk - 1) / sh.chunk) : 0;
      P.desc[cta * 2] = cut ? cut_at : make_int4(0, 0, 0, 0);
      P.desc[cta * 2 + 1] = make_int4(more, 0, 0, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh.dead) {  // a wait ran out: NaN for every row of this CTA's parts
    Walk k = sh.start;
    for (int seg = 0; k.next(P); ++seg) {
      const bool whole = k.j0 == 0 && k.j1 == k.s.J;
      const int slot = cta * 2 + (seg == 0 ? 0 : 1), from = k.u * 2 * P.npt;
      const int rows = min(k.s.n - from, 2 * P.npt) * P.G;
      for (int i = tid; i < rows; i += kThreads) {
        const int64_t row = static_cast<int64_t>(k.s.lo + from + i / P.G) * P.Hq + k.h * P.G + i % P.G;
        if (whole) {
          for (int e = 0; e < P.D; ++e) static_cast<uint16_t*>(P.out)[row * P.D + e] = 0x7FFF;
          if (P.lse) P.lse[row] = NAN;
        } else {
          const int tile = i / (P.npt * P.G);
          P.part_s[static_cast<int64_t>(slot * 2 + tile) * kTile + i - tile * P.npt * P.G] = make_float2(0.0f, NAN);
        }
      }
      if (tid == 0) {
        const bool cut = k.j0 == 0 && k.j1 < k.s.J;
        P.desc[cta * 2] = cut ? make_int4(k.s.lo + from, min(k.s.n - from, 2 * P.npt), k.h, slot) : make_int4(0, 0, 0, 0);
        P.desc[cta * 2 + 1] = make_int4(cut ? static_cast<int>((k.s.J - k.j1 + sh.chunk - 1) / sh.chunk) : 0, 0, 0, 0);
      }
    }
  }
  if (warp == kWarpS)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Join of the units that CTA borders cut.  Every block lists the cut units
// (one for each CTA at most) and takes its share of their items: 32 rows, a
// warp an eighth of the columns, or, where a unit has eight parts or more, 32
// rows by one group of four columns, a warp an eighth of the parts.  (26 nodes of
// 8 heads, the whole call, parts split over warps / not: 37 parts a unit 95 / 98
// us, 18: 96 / 95, 9: 175 / 173, 5: 183 / 178, 2: 232 / 185.)  Bound by the parts'
// bytes, so a lane has several loads in flight; parts are added in a fixed order.
constexpr int kJoinThreads = 256;

// Adds parts p, p + step, ... (kAt of them at a time, loaded together) of kGroups column groups;
// the shift follows the largest so far.
template <int kGroups, int kAt, typename Row>
__device__ __forceinline__ void join_parts(const AttnParams& P, Row row_of, int p, int parts, int step, int r,
                                           int cg, float& top, float& sum, float4 (&o)[kGroups]) {
  for (; p < parts; p += kAt * step) {
    float2 s[kAt];
    float4 x[kAt][kGroups];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      s[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) x[i][g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p + i * step < parts) {
        const int64_t tile = row_of(p + i * step);  // tile of the partial results
        s[i] = P.part_s[tile * kTile + r];
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
          x[i][g] = reinterpret_cast<const float4*>(P.part_o)[(tile * P.groups + cg + g) * kTile + r];
      }
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < kAt; ++i) now = fmaxf(now, s[i].x);
    const float f0 = top == -INFINITY ? 0.0f : ex2_approx(top - now);
    top = now;
    sum *= f0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) o[g] = make_float4(o[g].x * f0, o[g].y * f0, o[g].z * f0, o[g].w * f0);
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const float f = s[i].x == -INFINITY ? 0.0f : ex2_approx(s[i].x - top);
      sum += f * s[i].y;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        o[g].x += f * x[i][g].x;
        o[g].y += f * x[i][g].y;
        o[g].z += f * x[i][g].z;
        o[g].w += f * x[i][g].w;
      }
    }
  }
}

template <int DP, bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const __grid_constant__ AttnParams P) {
  __shared__ int first[kJoinThreads];   // first item behind each unit
  __shared__ int4 unit[kMaxCtas];
  __shared__ int parts_s[kMaxCtas];
  __shared__ int wsum[8];
  __shared__ float4 acc_s[8][32];
  __shared__ float2 st_s[8][32];
  constexpr int kGroups = DP / 32;  // column groups of a warp where it has all parts
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int last_row = P.npt * P.G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int items = 0;
  if (tid < P.ctas) {
    const int4 d = P.desc[tid * 2];
    const int parts = P.desc[tid * 2 + 1].x + 1;
    unit[tid] = d;
    parts_s[tid] = parts;
    const int blocks = d.y == 0 ? 0 : d.y > P.npt ? 4 + cdiv((d.y - P.npt) * P.G, 32) : cdiv(d.y * P.G, 32);
    items = blocks * (parts >= 8 ? DP / 4 : 1);
  }
  int incl = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  for (int i = 0; i < warp; ++i) incl += wsum[i];
  first[tid] = incl;
  __syncthreads();
  const int total = first[kJoinThreads - 1];
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = 0, hi = kJoinThreads - 1;  // the unit
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] > item) {
        hi = mid;
      } else {
        lo = mid + 1;
      }
    }
    const int cta = lo;
    const int4 d = unit[cta];
    const int parts = parts_s[cta];
    const int k = item - (cta > 0 ? first[cta - 1] : 0);
    const bool split = parts >= 8;
    const int rb = split ? k / (DP / 4) : k;
    const int tile = rb >> 2, r = (rb & 3) * 32 + lane;
    const int rnode = r / P.G, rg = r - rnode * P.G;
    const bool mine = r < last_row && tile * P.npt + rnode < d.y;
    const int64_t row = static_cast<int64_t>(d.x + tile * P.npt + rnode) * P.Hq + d.z * P.G + rg;
    auto at = [&](int p) { return static_cast<int64_t>((p == 0 ? d.w : (cta + p) * 2) * 2 + tile); };
    auto write = [&](int cg, float4 o, float inv) {
      if (cg * 4 < P.D)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + row * P.D + cg * 4) =
            make_uint2(pack2<kBf16>(o.x * inv, o.y * inv), pack2<kBf16>(o.z * inv, o.w * inv));
    };
    float top = -INFINITY, sum = 0.0f;
    if (!split) {
      float4 o[kGroups] = {};
      const int cg = warp * kGroups;
      if (mine) {
        join_parts<kGroups, 2>(P, at, 0, parts, 1, r, cg, top, sum, o);
        const float inv = inverse(sum);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) write(cg + g, o[g], inv);
        if (P.lse && warp == 0) P.lse[row] = (top + log2f(sum)) * kLn2;
      }
      continue;
    }
    float4 o[1] = {};
    const int cg = k - rb * (DP / 4);
    if (mine) join_parts<1, 4>(P, at, warp, parts, 8, r, cg, top, sum, o);
    acc_s[warp][lane] = o[0];
    st_s[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (warp == 0 && mine) {
      for (int i = 0; i < 8; ++i) top = fmaxf(top, st_s[i][lane].x);
      sum = 0.0f;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i = 0; i < 8; ++i) {
        const float2 s = st_s[i][lane];
        const float4 x = acc_s[i][lane];
        const float f = s.x == -INFINITY ? 0.0f : ex2_approx(s.x - top);
        sum += f * s.y;
        y.x += f * x.x;
        y.y += f * x.y;
        y.z += f * x.z;
        y.w += f * x.w;
      }
      const float inv = inverse(sum);
      write(cg, y, inv);
      if (P.lse && cg == 0) P.lse[row] = (top + log2f(sum)) * kLn2;
    }
    __syncthreads();
  }
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

template <int DP, bool kBf16>
int launch_attn(const AttnParams& p, int ctas, cudaStream_t stream) {
  constexpr size_t kSmem = Shape<DP>::kTiles + sizeof(Shared);
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  int rc = allow_smem(reinterpret_cast<const void*>(attn_kernel<DP, kBf16>), kSmem);
  if (rc != SV_OK) return rc;
  attn_kernel<DP, kBf16><<<ctas, kThreads, kSmem, stream>>>(p);
  if ((rc = check_launch("tree attention")) != SV_OK) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas * 4);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, combine_kernel<DP, kBf16>, p);
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
  const int ctas = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
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
  p.ctas = ctas;
  p.groups = (a->D <= 64 ? 64 : 128) / 4;
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

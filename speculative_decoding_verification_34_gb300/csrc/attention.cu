// Attention of a verification block (a chain or a draft tree) over the paged 8-bit cache.
//
// The target's forward over the drafts (tutorial §3.2) reads the whole cache once for a handful of rows: with G query
// heads to a kv head and n block rows, R = n * G rows share every key, out = softmax(scale * q.K^T) V.
//
// The keys and values go to the tensor cores as the e4m3 codes they are stored as, straight from TMA, and are never
// converted.  That needs the other operand in 8 bits without its rounding:
//   q   a bf16 number has 8 significant bits, an e4m3 number 4: after a power-of-two scale for each row q = hi + lo exactly
//       down to 2^-9 of the row's largest, and within 2^-17 of it below.  Both parts' products add up in one accumulator.
//   p   the weights are split into an e4m3 number and an e5m2 number for the rest: 7 bits of each weight, and, e5m2
//       having the exponents of half precision, weights down to 2^-27 of the reference value: the many small ones of
//       a long context beside one large one add up to something.
// Tokens are the other side of both products:
//     S^T [128 tokens, R] = K [128, D] . (qhi + qlo)^T        O^T [D, 2R] += V^T [D, 128] . [phi | plo]
// so every instruction has 128 full rows whatever R is, each thread of a warpgroup owns one token of a tile, its page's
// exponents are two factors of that thread (K's on its scores, V's on its weights), and the row sums stay in registers.
// The softmax's reference value is per row and for all tokens of an accumulator: it is the running maximum of score +
// V's exponent, raised (with the accumulator rescaled) only when a tile exceeds it by more than a factor 2^kSlack.  A row's
// first visible token sets it, however far below zero its score lies and whichever tile of the part it is in.
//
// A warp that walks a block's share publishes each item's part as a job before it loads its tiles, so the softmax warps
// stage the next job's queries while the last product of the one before is under way.
//
// Two persistent blocks to an SM, each one or two softmax warpgroups (sharing the rows where they are more than 32: 64
// scores and sums to a thread do not fit its registers), a warp that streams 128-token tiles (K, then V, a page at a
// time) into a ring of slots, and a warp that issues the products; one block's barriers, row setup and output overlap
// the other's arithmetic.  All tiles of all (sequence, kv head, row block) items are laid end to end and cut into equal
// shares, so ragged lengths balance; an item cut between blocks leaves unnormalised partials, which a second, dependent
// launch joins in a fixed order.
//
// Measured (GB300, 32 or 64 query heads, 8 kv heads of 128): 8 sequences of 50-65K tokens, 5 rows: 8 query heads to a kv
// head (40 rows) 170 us, 5.6 TB/s, bound by the softmax's chain for each tile; 4 or 1 to a kv head (20, 5 rows) 148, 151 us, 6.4,
// 6.3 TB/s, 0.94 of the measured copy rate.  64 sequences of 300-4091 tokens, 20 rows: 61 us, 4.9 TB/s (items of 3 to 33 tiles:
// their starts and ends, and blocks that end apart).  16 trees of 63 nodes at 700-2040 tokens, 256 rows: 82 us, 0.27 PFLOP/s of
// the operator's products: the softmax of four row blocks, an instruction issued in half of the cycles and no pipe full (the
// chain of one tile, barriers and all, with two tiles of an SM's two blocks to hide it).  One sequence of 505 tokens: 9.6 us,
// all latency.
// Measured and not kept: one block with two warpgroups on alternate tiles (batch 161 us: their row setup and output stopped
// both), weights as two e4m3 parts (range 2^-20, reference value raised in 61 % of the tiles), two tiles a step (batch 87 us:
// the ring holds too little ahead), partials joined by the last block to arrive (batch 69 us, and registers spilled), row
// blocks of 32 above 64 rows (trees 103 us: keys and values from the L2 twice as often).

#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>
#include <climits>
#include <cmath>

#include "kvcache.cuh"
#include "tree.cuh"

namespace specverify {
namespace {

constexpr int kTile = 128;                 // tokens of a tile: the M of a tcgen05 instruction
constexpr int kMaxGrid = 320;              // persistent blocks at most
constexpr int kItemCost = 4;               // what an item costs beside its tiles, in tiles (2: batch 68 us, 4: 65, 8: 66)
constexpr int kSlack = 5;                  // log2 by which weights may exceed 1 before their reference value is raised
constexpr float kPUnit = 8.f;              // weight 1 as an e4m3 operand: 8 * 2^kSlack = 256 <= 448
constexpr float kRest = 4096.f;            // scale of the weights' low parts: 8 * 4096 <= 57344, e5m2's largest
#ifndef SPEC_ATTENTION_WAIT_NS             // (shorter in a build that tests what follows)
#define SPEC_ATTENTION_WAIT_NS 2000000000
#endif
constexpr long long kWaitNs = SPEC_ATTENTION_WAIT_NS;    // bound on a wait for another role of the block
constexpr long long kDrainNs = 2000000000; // bound on a wait for copies and products in flight, before their memory is given up
constexpr int kMergeRows = 8;              // warps of a block of the joining launch

// An item that several blocks share, as the joining launch finds it.
struct __align__(16) SharedItem {
  int b, h, row0, live;                    // row0: the row block's first row
  int first, blocks;                       // the block that holds its first tile, how many share it (0: no such item)
  int pad[2];
};

struct AttnArgs {
  const __nv_bfloat16* q;
  int64_t qb, qn, qh;                      // strides of q
  __nv_bfloat16* out;
  const int8_t *ke, *ve;
  const int32_t *table, *kv_len, *num_draft, *parents;
  int32_t* status;
  int pages, max_pages, page, heads, group, B, gmax, root;
  bool q_vec;                              // q's rows may be read 8 bytes at a time
  float scale;                             // softmax scale * log2(e)
  float* part;                             // [2 * kMaxGrid][R][D]: unnormalised partial outputs
  float2* part_ml;                         // [2 * kMaxGrid][R]: their reference values and sums
  SharedItem* shared;              // [2][kMaxGrid]: the item that a block ends in and a later one goes on with; the one it goes on with
};

// --- PTX ------------------------------------------------------------------------------------------------------------

__device__ __forceinline__ unsigned smem(const void* p) { return unsigned(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint64_t* m, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem(m)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem(m)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* m, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem(m)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* m, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem(m)), "r"(parity)
      : "memory");
  return ok;
}
__device__ __forceinline__ bool mbar_test(uint64_t* m, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem(m)), "r"(parity)
      : "memory");
  return ok;
}
__device__ __forceinline__ long long now_ns() {
  long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// A bounded wait.  When it runs out it sets *dead and returns false, and no later wait of the block waits.  The block then
// comes to its end: the role that loads and the one that issues products stop at their next wait, the softmax goes on to the
// end of the job that it has taken, with accesses that stay in bounds whatever the data, and takes no other.  (A warp's lanes,
// and the softmax warps together, agree on that: their barriers need one another.)  What is in flight lands before its memory
// is given up, and every sequence of the block's share reports SPEC_ST_TIMEOUT: its rows may be unwritten, or joined from
// partials that are.  A try holds a thread for 4 us at most, so a tile costs little once no wait waits.
__device__ __forceinline__ bool mbar_wait(uint64_t* m, unsigned parity, volatile int* dead) {
  auto done = [&] { return kWaitNs < 4000 ? mbar_test(m, parity) : mbar_try(m, parity); };
  if (done()) return true;
  const long long t0 = now_ns();
  while (!done()) {
    if (*dead) return false;
    if (now_ns() - t0 > kWaitNs) {
      *dead = 1;
      return false;
    }
  }
  return true;
}
// Waits for what is in flight, whether or not the block gave up.
__device__ __forceinline__ void mbar_drain(uint64_t* m, unsigned parity) {
  const long long t0 = now_ns();
  while (!mbar_try(m, parity) && now_ns() - t0 < kDrainNs) {
  }
}
// A softmax warpgroup's own barrier (1 or 2), one that also says whether any of its threads has x, and one of all of them
// that says whether every thread has x.
template <int kId>
__device__ __forceinline__ void barrier_of() {
  asm volatile("barrier.cta.sync %0, 128;" ::"n"(kId) : "memory");
}
template <int kId>
__device__ __forceinline__ bool or_of(bool x) {
  unsigned r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n barrier.cta.red.or.pred p, %1, 128, q;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(r)
               : "n"(kId), "r"(unsigned(x))
               : "memory");
  return r;
}
template <int kGroups>
__device__ __forceinline__ void group_barrier(int grp) {
  if (kGroups == 1 || grp == 0)
    barrier_of<1>();
  else
    barrier_of<2>();
}
template <int kGroups>
__device__ __forceinline__ bool group_or(int grp, bool x) {
  return kGroups == 1 || grp == 0 ? or_of<1>(x) : or_of<2>(x);
}
template <int kCount>
__device__ __forceinline__ bool softmax_all(bool x) {
  unsigned r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n barrier.cta.red.and.pred p, 3, %1, q;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(r)
               : "n"(kCount), "r"(unsigned(x))
               : "memory");
  return r;
}
__device__ __forceinline__ void tma_page(const CUtensorMap* map, unsigned dst, uint64_t* bar, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem(bar)), "r"(0), "r"(y)
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* m) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem(m)) : "memory");
}
__device__ __forceinline__ void tc_mma(unsigned d, uint64_t a, uint64_t b, unsigned idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(unsigned(add))
      : "memory");
}
__device__ __forceinline__ void tc_load8(float (&x)[8], unsigned addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "r"(addr));
}
__device__ __forceinline__ void tc_store8(unsigned addr, const float (&x)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(x[0]), "f"(x[1]),
               "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory matrix descriptor: start, leading and stride byte offsets, swizzle (0 none, 2: 128 B, 4: 64 B).
__device__ __forceinline__ uint64_t matrix(unsigned addr, unsigned lbo, unsigned sbo, unsigned swizzle) {
  return uint64_t((addr & 0x3ffff) >> 4) | uint64_t(lbo >> 4) << 16 | uint64_t(sbo >> 4) << 32 | 1ull << 46 | uint64_t(swizzle) << 61;
}

// --- the shares of the work ------------------------------------------------------------------------------------------

// What one sequence asks for: rows of its block, tokens they may see, items (row blocks x kv heads) of kItemCost + tiles units.
struct Sequence {
  int rows, context, tokens, tiles, blocks;
  long long units;
};

template <int R>
__device__ __forceinline__ Sequence sequence(const AttnArgs& a, int b) {
  Sequence s;
  int n = a.num_draft ? a.num_draft[b] : a.gmax;
  n = min(max(n, 0), a.gmax);
  const int t = a.kv_len[b];
  s.rows = t < 0 ? 0 : n + a.root;
  s.context = t;
  const long long room = (long long)(a.max_pages) * a.page;
  s.tokens = int(min((long long)(t) + s.rows, room));
  s.tiles = s.rows ? (s.tokens + kTile - 1) / kTile : 0;
  s.blocks = (s.rows * a.group + R - 1) / R;
  s.units = s.rows ? (long long)(s.tiles + kItemCost) * (s.blocks * a.heads) : 0;
  return s;
}

// A block's part of one item: tiles [tile, tile + count) of (b, h, row block rb).
struct Job {
  int b, h, rb, tile, count;               // count 0: no more
  int tokens, tiles, context;              // the sequence's tokens and tiles, those of the tokens before the block
  int live;                                // rows of the row block
  int starts, ends;                        // whether the item's first, last tile are among them
  int first, blocks;                       // where not both: the block that holds the item's first tile, how many share it
};

// Walks a share of the units, an item after another.  An item's first kItemCost units stand for no tile.
template <int R>
struct Walk {
  int b;
  long long at, left;                      // unit within sequence b, units of the share still to come
  Sequence s;
  __device__ __forceinline__ Walk(const AttnArgs& a, int b_, long long at_, long long left_)
      : b(b_), at(at_), left(left_), s(sequence<R>(a, b_)) {}
  // `end`: the share's end among all units; owner(u): the block whose share holds unit u.
  template <class Owner>
  __device__ __forceinline__ Job next(const AttnArgs& a, long long end, Owner owner) {
    Job g{};
    while (left > 0) {
      while (at >= s.units) {              // sequences without work, or the share goes on in the next one
        at -= s.units;
        s = sequence<R>(a, ++b);
      }
      const int each = s.tiles + kItemCost;
      const int item = at < UINT_MAX ? int(unsigned(at) / unsigned(each)) : int(at / each);
      const int from = int(at - (long long)(item) * each), to = int(min((long long)(each), from + left));
      at += to - from;
      left -= to - from;
      g.b = b;
      g.h = int(unsigned(item) / unsigned(s.blocks));
      g.rb = item - g.h * s.blocks;
      g.tile = max(from - kItemCost, 0);
      g.count = max(to - kItemCost, 0) - g.tile;
      g.tokens = s.tokens;
      g.tiles = s.tiles;
      g.context = s.context;
      g.live = min(R, s.rows * a.group - g.rb * R);
      g.starts = g.tile == 0;
      g.ends = to == each;
      if (g.count == 0) continue;
      if (!g.starts || !g.ends) {
        const long long u = end - left - to + kItemCost;   // the unit of the item's first tile
        g.first = owner(u);
        g.blocks = owner(u + s.tiles - 1) - g.first + 1;
      }
      return g;
    }
    g.count = 0;
    return g;
  }
};

template <int R, int D>
struct Layout {
  static constexpr int kGroups = R > 32 ? 2 : 1;          // softmax warpgroups, each with R / kGroups of the rows
  static constexpr int kRows = R / kGroups;
  static constexpr int kSoft = 128 * kGroups, kThreads = kSoft + 64;
  static constexpr int kNP = (R + 15) / 16 * 16;          // columns of the scores, and of each part of the weights
  static constexpr int kSide = kTile * D;                 // bytes of a K or V tile: a slot of the ring
  static constexpr int kQ = 2 * kNP * D, kP = 2 * kNP * kTile; // bytes
  static constexpr int kFixed = kQ + kP + 1024 + 4096 + 60 * R;     // with room to align to 1024, and Shared
  static constexpr int kSlots = (115712 - kFixed) / kSide < 10 ? (115712 - kFixed) / kSide : 10;     // half an SM's memory
  static constexpr int kRing = kSlots * kSide;
  static constexpr int kBytes = kRing + kQ + kP + 1024;
  static constexpr int kColumns = 3 * kNP <= 64 ? 64 : 3 * kNP <= 128 ? 128 : 256;
  static constexpr unsigned kSwizzle = D == 128 ? 2 : 4;
  static constexpr unsigned kAtom = 8 * D;                // eight rows of a swizzled tile
  static_assert(kRows % 8 == 0 && R <= 64, "eight rows are loaded at once, 64 fit a mask");
};

constexpr int kJobs = 3;                   // jobs published at a time

template <int R, int kSlots>
struct __align__(16) Shared {
  float qf[2][R], ref[2][R];               // of this job and the next: factor on a row's scores, minus its reference value
  float peak[4][R];                        // per warp: largest score of a row, then its sum
  float f[R], fall[R];                     // rise of a row's reference value, then factor on its outputs; factor on what it has so far
  int unset[R];                            // the row has seen no token yet
  int head[2][R];                          // a row's place in a sequence's block: row * Hq + head
  unsigned long long path[64], seen[kJobs][64];     // rows of the row block that see a token of the block, a bit each
  Job job[kJobs];
  int up[64];
  int slot[kSlots][8];                     // pages of a V slot's tile: exponents of K and V, or kNoPage
  uint64_t full[kSlots], empty[kSlots], job_full[kJobs], seen_full[kJobs], job_empty[kJobs];
  uint64_t s_full, s_free, p_ready, pv_done, q_ready, drained;
  unsigned tmem;
  int dead;                                // a wait ran out
  long long scan[10];
  int start_b;                             // the share: its first sequence, the first unit of that, units
  long long start_at, share;
};
constexpr int kNoPage = INT_MIN;

// Two products, sums, or products added to something, in one instruction.
__device__ __forceinline__ uint64_t both(float2 a) { return uint64_t(__float_as_uint(a.x)) | uint64_t(__float_as_uint(a.y)) << 32; }
__device__ __forceinline__ float2 both(uint64_t a) { return make_float2(__uint_as_float(unsigned(a)), __uint_as_float(unsigned(a >> 32))); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(both(a)), "l"(both(b)));
  return both(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(both(a)), "l"(both(b)));
  return both(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(both(a)), "l"(both(b)), "l"(both(c)));
  return both(r);
}

// The largest of a warp's 32 values.
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// Sums over a warp of R values a thread: lane l with l % 4 == 0 writes those of rows 8k + {4, 2, 1} . bits {4, 3, 2} of l.
template <int R>
__device__ __forceinline__ void warp_sums(const float2 (&pairs)[R / 2], float* to) {
  float x[R];
#pragma unroll
  for (int r = 0; r < R; r += 2) x[r] = pairs[r / 2].x, x[r + 1] = pairs[r / 2].y;
  const int lane = int(threadIdx.x) & 31;
#pragma unroll
  for (int k = 0; k < R; k += 8) {
    float y[4], z[2], w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float keep = lane & 16 ? x[k + i + 4] : x[k + i], give = lane & 16 ? x[k + i] : x[k + i + 4];
      y[i] = keep + __shfl_xor_sync(~0u, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float keep = lane & 8 ? y[i + 2] : y[i], give = lane & 8 ? y[i] : y[i + 2];
      z[i] = keep + __shfl_xor_sync(~0u, give, 8);
    }
    const float keep = lane & 4 ? z[1] : z[0], give = lane & 4 ? z[0] : z[1];
    w = keep + __shfl_xor_sync(~0u, give, 4);
    w += __shfl_xor_sync(~0u, w, 2);
    w += __shfl_xor_sync(~0u, w, 1);
    if ((lane & 3) == 0) to[k + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1)] = w;
  }
}

// Two weights: e4m3 high parts, e5m2 low parts.  In half precision: 11 bits of a weight, of which the parts keep 7.
__device__ __forceinline__ void split_pair(float2 x, unsigned& hi, unsigned& lo) {
  const __half2 p = __floats2half2_rn(x.x, x.y);
  const __half2_raw raw = p;
  hi = __nv_cvt_halfraw2_to_fp8x2(raw, __NV_SATFINITE, __NV_E4M3);
  const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(hi), __NV_E4M3));
  const __half2_raw rest = __hmul2(__hsub2(p, h), __float2half2_rn(kRest));
  lo = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E5M2);
}

// A job's queries go to shared memory as two e4m3 operands, in the layout that TMA gives the keys; row r is warp
// r % kWarps's, and the loads of a warp's rows are all in flight before the first is used.
template <int R, int D>
struct Queries {
  static constexpr int kWarps = Layout<R, D>::kSoft / 32, kEach = R / kWarps, kWords = D / 64;
  unsigned raw[kEach][kWords];                             // kWords pairs of bf16 a lane

  __device__ __forceinline__ void load(const AttnArgs& a, const Job& g, int* heads) {
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    // lane k divides for row k * kWarps + warp: its place in the block, and its element in q
    const unsigned row = unsigned(g.rb * R + lane * kWarps + warp), i = row / unsigned(a.group);
    const unsigned h = g.h * a.group + (row - i * a.group), place = i * a.heads * a.group + h;
    const long long element = g.b * a.qb + i * a.qn + h * a.qh;
    if (lane < kEach && lane * kWarps + warp < g.live) heads[lane * kWarps + warp] = int(place);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) raw[k][w] = 0;
      const __nv_bfloat16* q = a.q + __shfl_sync(~0u, element, k) + lane * 2 * kWords;
      if (k * kWarps + warp < g.live) {
        if (a.q_vec) {
          if constexpr (kWords == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(q);
            raw[k][0] = x.x, raw[k][1] = x.y;
          } else {
            raw[k][0] = *reinterpret_cast<const unsigned*>(q);
          }
        } else {
#pragma unroll
          for (int w = 0; w < kWords; ++w)
            raw[k][w] = unsigned(__bfloat16_as_ushort(q[2 * w])) | unsigned(__bfloat16_as_ushort(q[2 * w + 1])) << 16;
        }
      }
    }
  }

  __device__ __forceinline__ void put(const AttnArgs& a, const Job& g, uint8_t* q_smem, float* qf, float* ref) {
    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    // the largest |x| of each row, as bf16 bits (all rows' at once: each is a chain of its own)
    unsigned tops[kEach], most = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      unsigned top = raw[k][0] & 0x7fff7fffu;
#pragma unroll
      for (int w = 1; w < kWords; ++w) top = __vmaxu2(top, raw[k][w] & 0x7fff7fffu);
      tops[k] = __reduce_max_sync(~0u, max(top >> 16, top & 0xffffu));
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) most = max(most, tops[k]);
    if (most >= 0x7f80u) {                                 // an infinite or NaN query: NaN in its place, the others scaled
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        unsigned top = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          unsigned x = raw[k][w];
          const unsigned lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
          if (lo < 0x7f80u) top = max(top, lo); else x |= 0x7fffu;
          if (hi < 0x7f80u) top = max(top, hi); else x |= 0x7fff0000u;
          raw[k][w] = x;
        }
        tops[k] = __reduce_max_sync(~0u, top);
      }
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int r = k * kWarps + warp;
      const unsigned top = tops[k];
      // it goes to [128, 256)
      const int s = min(7 - max(int(top >> 7) - 127, -126), 120);
      const float up = pow2(s);
      unsigned hi = 0, lo = 0;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const __half2 x = __floats2half2_rn(__uint_as_float(raw[k][w] << 16) * up, __uint_as_float(raw[k][w] & 0xffff0000u) * up);
        const __half2_raw xr = x;
        const unsigned h = __nv_cvt_halfraw2_to_fp8x2(xr, __NV_SATFINITE, __NV_E4M3);
        const __half2 back = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(h), __NV_E4M3));
        const __half2_raw rest = __hsub2(x, back);
        hi |= h << (16 * w);
        lo |= unsigned(__nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3)) << (16 * w);
      }
      // D = 128: four bytes a lane, 16-byte chunk ^ row % 8; D = 64: two bytes, chunk ^ (row / 2) % 4
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int n = part * Layout<R, D>::kNP + r;
        const unsigned byte = unsigned(lane * 2 * kWords), chunk = byte >> 4, at = byte & 15;
        uint8_t* dst = q_smem + n * D + ((chunk ^ (D == 128 ? n & 7 : (n >> 1) & 3)) << 4) + at;
        if constexpr (kWords == 2)
          *reinterpret_cast<unsigned*>(dst) = part ? lo : hi;
        else
          *reinterpret_cast<unsigned short*>(dst) = (unsigned short)(part ? lo : hi);
      }
      if (lane == 0) qf[r] = r < g.live ? pow2(-s) * a.scale : 0.f, ref[r] = 0.f;
    }
  }
};

template <int R, int D>
__global__ void __launch_bounds__(Layout<R, D>::kThreads, 2)
    attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using L = Layout<R, D>;
  constexpr int kSlots = L::kSlots, kNP = L::kNP, kThreads = L::kThreads;
  constexpr int kTmaWarp = L::kSoft / 32, kMmaWarp = kTmaWarp + 1;
  static_assert(kSlots >= 4, "two tiles at least");
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared<R, kSlots> sh;
  static_assert(L::kBytes + sizeof(sh) <= 115712, "half the shared memory of an SM");
  uint8_t* const ring = raw_smem + ((1024 - (smem(raw_smem) & 1023)) & 1023);
  uint8_t* const q_smem = ring + L::kRing;
  uint8_t* const p_smem = q_smem + L::kQ;
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.s_full, 1);
    mbar_init(&sh.s_free, L::kSoft);
    mbar_init(&sh.p_ready, L::kSoft);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.q_ready, L::kSoft);
    mbar_init(&sh.drained, 1);
    for (int i = 0; i < kJobs; ++i) {
      mbar_init(&sh.job_full[i], 1);
      mbar_init(&sh.seen_full[i], 1);
      mbar_init(&sh.job_empty[i], 2);
    }
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_launches_before();
  // the share of this block: the sequences' units are summed, then the one that holds the share's first unit is found
  const int me = int(blockIdx.x);
  long long total = 0, mine = 0, up_to = 0;                // units of all, of this thread's sequence, up to and with it
  auto scan = [&](int b) {
    mine = b < a.B ? sequence<R>(a, b).units : 0;
    up_to = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(~0u, up_to, o);
      if (lane >= o) up_to += t;
    }
    __syncthreads();
    if (lane == 31) sh.scan[warp] = up_to;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) up_to += sh.scan[w];
      all += sh.scan[w];
    }
    return all;
  };
  for (int b0 = 0; b0 < a.B; b0 += kThreads) total += scan(b0 + tid);
  const int blocks = int(min((long long)(gridDim.x), total));
  if (tid == 0) a.shared[me].blocks = a.shared[kMaxGrid + me].blocks = 0;
  // Counts out of range, also of sequences without rows, which no job meets: block 0 reports them, once its tiles are on their way.
  auto report_counts = [&]() {
    if (me > 0 || !a.status || !a.num_draft) return;
    for (int b = lane; b < a.B; b += 32)
      if (a.num_draft[b] < 0 || a.num_draft[b] > a.gmax) atomicOr(a.status + b, SPEC_ST_CLAMPED_GAMMA);
  };
  if (me >= blocks) {                                      // (block 0: nobody has rows)
    if (warp == 0) report_counts();
    return;
  }
  const long long first = total * me / blocks;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const long long all = a.B <= kThreads ? 0 : scan(b0 + tid);
    if (before + up_to - mine <= first && first < before + up_to) {
      sh.start_b = b0 + tid;
      sh.start_at = first - (before + up_to - mine);
    }
    before += all;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem(&sh.tmem)), "n"(L::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before();
  }
  __syncthreads();
  tc_after();
  let_next_start();
  const unsigned tmem = sh.tmem;
  volatile int* const dead = &sh.dead;

  if (warp == kTmaWarp) {
    // --- jobs, and their tiles into the ring, a page at a time; lane l keeps page l of a window of 32 pages --------------
    const long long end = total * (me + 1) / blocks;
    Walk<R> walk(a, sh.start_b, sh.start_at, end - first);
    if (lane == 0) sh.share = end - first;
    auto owner = [&](long long u) { return int(((u + 1) * blocks - 1) / total); };
    const int per = kTile / a.page;                       // pages of a tile
    unsigned filled = 0, slot = 0, turn = 0;              // slots so far; the next one and how often the ring went round
    bool gone = false;
    for (unsigned jobs = 0; !gone; ++jobs) {
      const Job g = walk.next(a, end, owner);
      if (g.blocks && lane == 0)
        a.shared[(g.starts ? 0 : kMaxGrid) + me] = SharedItem{g.b, g.h, g.rb * R, g.live, g.first, g.blocks, {0, 0}};
      const unsigned js = jobs % kJobs;
      if (jobs >= kJobs && __any_sync(~0u, !mbar_wait(&sh.job_empty[js], (jobs / kJobs - 1) & 1, dead))) break;
      if (lane == 0) {
        sh.job[js] = g;
        mbar_arrive(&sh.job_full[js]);
      }
      if (g.count == 0) break;
      // its queries come to the L2 while the softmax is at the tiles before
      for (int i = lane; i < g.live * (D / 64); i += 32) {
        const unsigned row = unsigned(g.rb * R + i / (D / 64)), at = row / unsigned(a.group);
        const __nv_bfloat16* q = a.q + g.b * a.qb + at * a.qn + (g.h * a.group + (row - at * a.group)) * a.qh;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i % (D / 64) * 64));
      }
      const int p_end = (g.tokens + a.page - 1) / a.page;                    // pages of the sequence that hold tokens
      const int32_t* table = a.table + int64_t(g.b) * a.max_pages;
      int p0 = g.tile * per;
      const int last = min((g.tile + g.count) * per, p_end);
      auto page_of = [&](int p) { return p + lane < last ? table[p + lane] : -1; };
      auto exps_of = [&](int pid) {
        if (pid < 0 || pid >= a.pages) return kNoPage;
        const int64_t row = int64_t(pid) * a.heads + g.h;
        return (stored_exponent(a.ke[row]) << 8) | (stored_exponent(a.ve[row]) & 0xff);
      };
      int pid = page_of(p0), exps = exps_of(pid);
      int next_pid = page_of(p0 + 32), next_exps = kNoPage;
      bool bad = p0 + lane < last && exps == kNoPage;
      for (int i = 0; i < g.count; ++i) {
        const int here = (g.tile + i) * per - p0;                            // the tile's pages are lanes [here, here + per)
        const bool own = lane >= here && lane < here + per;
        const bool load = own && exps != kNoPage;
        const unsigned bytes = unsigned(__popc(__ballot_sync(~0u, load)) * a.page * D);
        const int y = (pid * a.heads + g.h) * a.page;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          gone = __any_sync(~0u, turn && !mbar_wait(&sh.empty[slot], (turn - 1) & 1, dead));
          if (gone) break;                                  // the slot may still be filled or read
          if (side && own) sh.slot[slot][lane - here] = exps;
          __syncwarp();
          if (lane == 0) mbar_expect(&sh.full[slot], bytes);
          __syncwarp();
          if (load)
            tma_page(side ? &map_v : &map_k, smem(ring + slot * L::kSide) + unsigned((lane - here) * a.page * D),
                     &sh.full[slot], y);
          if (++slot == kSlots) slot = 0, ++turn;
          ++filled;
        }
        if (gone) break;
        if (here == 0) next_exps = exps_of(next_pid);
        if (here + per == 32) {
          p0 += 32;
          pid = next_pid, exps = next_exps;
          bad |= p0 + lane < last && exps == kNoPage;
          next_pid = page_of(p0 + 32);
        }
        if (i == 0) {
          // which rows see a token of the block; waited for where a tile holds one
          int nd = a.num_draft ? a.num_draft[g.b] : a.gmax;
          int bits = 0;
          nd = min(max(nd, 0), a.gmax);
          const unsigned long long all = g.live == 64 ? ~0ull : (1ull << g.live) - 1;
          if (a.parents == nullptr) {
            for (int j = lane; j < 64; j += 32) {          // block row i sees token j <= i; rows from j * group on
              const int r = j * a.group - g.rb * R;
              sh.seen[js][j] = r <= 0 ? all : r >= 64 ? 0ull : all & (~0ull << r);
            }
          } else {
            if (path_masks(a.parents + int64_t(g.b) * a.gmax, nd, sh.path, sh.up)) bits |= SPEC_ST_BAD_TREE;
            unsigned long long m[2] = {0, 0};
            int row = (g.rb * R) / a.group, left = a.group - (g.rb * R) % a.group;
            for (int r = 0; r < g.live; ++r) {
              const unsigned long long sees = a.root ? (sh.path[row] << 1) | 1 : sh.path[row + 1];
              m[0] |= ((sees >> lane) & 1) << r;
              m[1] |= ((sees >> (lane + 32)) & 1) << r;
              if (--left == 0) ++row, left = a.group;
            }
            sh.seen[js][lane] = m[0], sh.seen[js][lane + 32] = m[1];
          }
          if ((long long)(g.context) + nd + a.root > g.tokens) bits |= SPEC_ST_BAD_PAGE;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.seen_full[js]);
            if (bits && a.status) atomicOr(a.status + g.b, bits);
          }
        }
      }
      if (bad && a.status) atomicOr(a.status + g.b, SPEC_ST_BAD_PAGE);
    }
    report_counts();
    // the copies in flight land before the block may end
    for (unsigned k = 0; k < kSlots && k < filled; ++k) {
      turn -= slot == 0;
      slot = slot == 0 ? kSlots - 1 : slot - 1;
      mbar_drain(&sh.full[slot], turn & 1);
    }
  } else if (warp == kMmaWarp) {
    // --- MMA: one thread issues both products ---------------------------------------------------------------------------
    if (lane == 0) {
      // A: tokens (K-major) or D (M-major: bit 15), B: columns (K-major) or (N-major: bit 16); f32 accumulators
      constexpr unsigned kS = 1u << 4 | unsigned(kNP >> 3) << 17 | unsigned(kTile >> 4) << 24;
      constexpr unsigned kHi = 1u << 4 | 1u << 15 | 1u << 16 | unsigned(kNP >> 3) << 17 | unsigned(D >> 4) << 24;
      constexpr unsigned kRest5 = kHi | 1u << 10;          // B is e5m2
      const unsigned q0 = smem(q_smem), p0 = smem(p_smem);
      unsigned n_s = 0, n_p = 0;                           // score products, output products issued
      for (unsigned jobs = 0;; ++jobs) {
        const unsigned js = jobs % kJobs;
        if (!mbar_wait(&sh.job_full[js], (jobs / kJobs) & 1, dead) || *dead) break;
        const int count = sh.job[js].count;
        if (count == 0) break;
        mbar_arrive(&sh.job_empty[js]);
        if (!mbar_wait(&sh.q_ready, jobs & 1, dead)) break;
        const unsigned end = n_p + unsigned(count), begin = n_p;
        long long t0 = now_ns();
        for (unsigned poll = 1; n_p < end; ++poll) {
          // scores of the next tile: its keys are there and the last scores have been read
          const unsigned ks = (2 * n_s) % kSlots, kt = (2 * n_s) / kSlots;
          if (n_s < end && n_s <= n_p + 1 && mbar_test(&sh.full[ks], kt & 1) &&
              (n_s == 0 || mbar_test(&sh.s_free, (n_s - 1) & 1))) {
            tc_after();
            const unsigned k0 = smem(ring + ks * L::kSide);
#pragma unroll
            for (int k = 0; k < 2 * D / 32; ++k) {         // the queries' high parts, then their low parts
              const unsigned at = (k % (D / 32)) * 32, part = k / (D / 32) * kNP * D;
              tc_mma(tmem, matrix(k0 + at, 16, L::kAtom, L::kSwizzle), matrix(q0 + part + at, 16, L::kAtom, L::kSwizzle), kS, k > 0);
            }
            tc_commit(&sh.s_full);
            tc_commit(&sh.empty[ks]);
            ++n_s;
            poll = 0;
          }
          // outputs of a tile whose weights are written
          const unsigned vs = (2 * n_p + 1) % kSlots;
          if (n_p < n_s && mbar_test(&sh.p_ready, n_p & 1) && mbar_test(&sh.full[vs], ((2 * n_p + 1) / kSlots) & 1)) {
            tc_after();
            const unsigned v0 = smem(ring + vs * L::kSide);
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k) {
              const uint64_t v = matrix(v0 + k * 32 * D, L::kAtom, L::kAtom, L::kSwizzle);
              const bool add = k > 0 || n_p > begin;
              tc_mma(tmem + kNP, v, matrix(p0 + k * 32 * 16, 128, kTile * 16, 0), kHi, add);
              tc_mma(tmem + 2 * kNP, v, matrix(p0 + kNP * kTile + k * 32 * 16, 128, kTile * 16, 0), kRest5, add);
            }
            tc_commit(&sh.empty[vs]);
            tc_commit(&sh.pv_done);
            ++n_p;
            poll = 0;
          }
          if (poll == 0) {
            t0 = now_ns();
          } else if ((poll & 255) == 0 && (*dead || now_ns() - t0 > kWaitNs)) {
            *dead = 1;
            break;
          }
        }
        if (n_p < end) break;
      }
    }
    __syncwarp();
  } else {
    // --- softmax: a thread for each token of a tile ---------------------------------------------------------------------
    constexpr int RT = L::kRows;                           // rows of this warpgroup: [c0, c0 + RT)
    const int t = tid & 127, quad = warp & 3, grp = warp >> 2, c0 = grp * RT;
    const unsigned lanes = tmem + (unsigned(quad * 32) << 16), o_tm = lanes + kNP + c0;
    uint8_t* const p_mine = p_smem + t * 16;
    const int page_shift = 31 - __clz(a.page);
    unsigned n = 0, v_slot = 1, v_turn = 0;                // tiles so far; the slot of the next V and how often the ring went round
    const bool any = __all_sync(~0u, mbar_wait(&sh.job_full[0], 0, dead) && sh.job[0].count > 0);
    if (any) {
      Queries<R, D> q;
      q.load(a, sh.job[0], sh.head[0]);
      q.put(a, sh.job[0], q_smem, sh.qf[0], sh.ref[0]);
    }
    fence_async_smem();
    tc_before();
    bool go = softmax_all<L::kSoft>(any);                  // (the same in all softmax threads: they meet the same barriers)
    mbar_arrive(&sh.q_ready);
    for (unsigned jobs = 0; go; ++jobs) {
      const unsigned js = jobs % kJobs;
      const Job& g = sh.job[js];
      const int count = g.count;
      const float* const qf = sh.qf[jobs & 1] + c0;
      float* const ref = sh.ref[jobs & 1] + c0;
      float2 sum[RT / 2];                                  // of rows 2i and 2i + 1
#pragma unroll
      for (int r = 0; r < RT / 2; ++r) sum[r] = make_float2(0.f, 0.f);
      bool open = true;                                    // a row of the warpgroup is unset
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        mbar_wait(&sh.full[v_slot], v_turn & 1, dead);
        const int tile = (g.tile + i) * kTile;
        const int exps = sh.slot[v_slot][t >> page_shift];
        const bool valid = tile + t < g.tokens && exps != kNoPage;
        const float kf = valid ? pow2(exps >> 8) : 0.f;
        const int ev = valid ? int(int8_t(exps & 0xff)) : 0;
        if (!valid && grp == 0) {                          // what no token was written to must not reach the product
          uint8_t* const v_row = ring + v_slot * L::kSide + t * D;
#pragma unroll
          for (int c = 0; c < D; c += 16) *reinterpret_cast<uint4*>(v_row + c) = make_uint4(0, 0, 0, 0);
        }
        v_slot += 2;
        if (v_slot >= kSlots) v_slot -= kSlots, ++v_turn;
        mbar_wait(&sh.s_full, n & 1, dead);
        tc_after();
        float2 x[RT / 2];                                  // of rows 2i and 2i + 1
        {
          float s8[RT / 8][8];
#pragma unroll
          for (int c = 0; c < RT / 8; ++c) tc_load8(s8[c], lanes + c0 + c * 8);
          tc_wait_ld();
#pragma unroll
          for (int r = 0; r < RT / 2; ++r) x[r] = make_float2(s8[r / 4][r % 4 * 2], s8[r / 4][r % 4 * 2 + 1]);
        }
        tc_before();
        mbar_arrive(&sh.s_free);
        // log2 of the weights, relative to each row's reference value
#pragma unroll
        for (int r = 0; r < RT; r += 4) {
          const float4 f = *reinterpret_cast<const float4*>(qf + r), m = *reinterpret_cast<const float4*>(ref + r);
          const float2 k2 = make_float2(kf, kf);
          x[r / 2] = fma2(x[r / 2], mul2(make_float2(f.x, f.y), k2), make_float2(m.x, m.y));
          x[r / 2 + 1] = fma2(x[r / 2 + 1], mul2(make_float2(f.z, f.w), k2), make_float2(m.z, m.w));
        }
        if (tile + kTile > g.context || !valid) {          // tokens of the block, or none
          mbar_wait(&sh.seen_full[js], (jobs / kJobs) & 1, dead);
          const int j = tile + t - g.context;
          const unsigned sees = unsigned((!valid ? 0ull : j < 0 ? ~0ull : sh.seen[js][j]) >> c0);
#pragma unroll
          for (int r = 0; r < RT / 2; ++r) {
            if (!((sees >> (2 * r)) & 1)) x[r].x = -INFINITY;
            if (!((sees >> (2 * r + 1)) & 1)) x[r].y = -INFINITY;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < RT / 2; ++r) top = fmaxf(top, fmaxf(x[r].x, x[r].y));
        if (group_or<L::kGroups>(grp, open || top + float(ev) > float(kSlack))) {
          // a row's reference value rises to the tile's largest score + V's exponent; an unset one becomes that, whatever
          // its sign, and stays 0 while the tiles show the row nothing (-inf; a NaN row counts as set)
          float up = 0.f;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float m = warp_max((r & 1 ? x[r / 2].y : x[r / 2].x) + float(ev));
            if (lane == r) up = m;
          }
          if (lane < RT) sh.peak[quad][c0 + lane] = up;
          group_barrier<L::kGroups>(grp);
          bool unset = false;
          if (t < RT) {
            const int r = c0 + t;
            up = fmaxf(fmaxf(sh.peak[0][r], sh.peak[1][r]), fmaxf(sh.peak[2][r], sh.peak[3][r]));
            unset = i == 0 || sh.unset[r];
            const float rise = unset && up > -INFINITY ? up : fmaxf(up, 0.f);
            unset = unset && up == -INFINITY;
            sh.unset[r] = unset;
            sh.f[r] = rise;
            sh.fall[r] = ex2(fminf(-rise, 0.f));           // (a row that was unset has nothing so far)
            ref[t] -= rise;
          }
          if (i > 0) mbar_wait(&sh.pv_done, (n - 1) & 1, dead);
          open = group_or<L::kGroups>(grp, unset);
          tc_after();
#pragma unroll
          for (int r = 0; r < RT; r += 8) {
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 rise = *reinterpret_cast<const float2*>(sh.f + c0 + r + 2 * e);
              x[r / 2 + e].x -= rise.x;
              x[r / 2 + e].y -= rise.y;
              most = fmaxf(most, fmaxf(rise.x, rise.y));
            }
            if (i > 0 && most > 0.f) {                     // (the same in every thread)
              float hi[8], lo[8];
              tc_load8(hi, o_tm + r);
              tc_load8(lo, o_tm + kNP + r);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = *reinterpret_cast<const float2*>(sh.fall + c0 + r + 2 * e);
                sum[r / 2 + e] = mul2(sum[r / 2 + e], f);
                hi[2 * e] *= f.x, hi[2 * e + 1] *= f.y;
                lo[2 * e] *= f.x, lo[2 * e + 1] *= f.y;
              }
              tc_store8(o_tm + r, hi);
              tc_store8(o_tm + kNP + r, lo);
            }
          }
          if (i > 0) tc_wait_st();
        } else {
          mbar_wait(&sh.pv_done, (n - 1) & 1, dead);       // the product that reads the last weights is done
        }
        ++n;
        const float vf = pow2(ev) * kPUnit;
#pragma unroll
        for (int r = 0; r < RT; r += 8) {
          unsigned hi[2], lo[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            unsigned h[2], l[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = r / 2 + c * 2 + e;
              const float2 u = make_float2(ex2(x[at].x), ex2(x[at].y));
              sum[at] = add2(sum[at], u);
              split_pair(mul2(u, make_float2(vf, vf)), h[e], l[e]);
            }
            hi[c] = h[0] | h[1] << 16;
            lo[c] = l[0] | l[1] << 16;
          }
          // eight columns of 16: column m of token t is byte m % 16 of vector t of group m / 16
          uint8_t* const to = p_mine + ((c0 + r) >> 4) * (kTile * 16) + ((c0 + r) & 8);
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + kNP * kTile) = make_uint2(lo[0], lo[1]);
        }
        fence_async_smem();
        tc_before();
        mbar_arrive(&sh.p_ready);
      }

      // --- the next job's queries: their shared memory is free, all score products of this job are done ---------------------
      const unsigned ns = (jobs + 1) % kJobs;
      const bool more = __all_sync(~0u, mbar_wait(&sh.job_full[ns], ((jobs + 1) / kJobs) & 1, dead) && sh.job[ns].count > 0);
      Queries<R, D> q;
      if (more) q.load(a, sh.job[ns], sh.head[(jobs + 1) & 1]);
      // --- the end of this one: the accumulator goes out, normalised or as a partial ---------------------------------------
      const bool whole = g.starts && g.ends;
      const int live = g.live;
      const int64_t place = int64_t(2 * me + (g.starts ? 1 : 0)) * R;
      warp_sums<RT>(sum, sh.peak[quad] + c0);
      if (more) q.put(a, sh.job[ns], q_smem, sh.qf[(jobs + 1) & 1], sh.ref[(jobs + 1) & 1]);
      fence_async_smem();
      group_barrier<L::kGroups>(grp);
      mbar_arrive(&sh.q_ready);
      if (t < RT) {
        const int r = c0 + t;
        const float all = sh.peak[0][r] + sh.peak[1][r] + sh.peak[2][r] + sh.peak[3][r];
        sh.f[r] = (whole ? (all == 0.f ? 0.f : 1.f / all) : 1.f) / kPUnit;
        if (!whole) a.part_ml[place + r] = make_float2(all == 0.f ? -INFINITY : -ref[t], all);
      }
      mbar_wait(&sh.pv_done, (n - 1) & 1, dead);
      group_barrier<L::kGroups>(grp);
      tc_after();
      const int d = D == 128 ? t : quad * 16 + lane;
      const bool has_d = D == 128 || lane < 16;
      __nv_bfloat16* const out = a.out + int64_t(g.b) * (a.gmax + a.root) * a.heads * a.group * D + d;
      float* const part = a.part + place * D + d;
      const int* const head = sh.head[jobs & 1];
      // rows read from the accumulator at once: two warpgroups' registers hold 8 (16: trees 84 -> 87 us), one's 16 or 24 (8: batch
      // 62.6 -> 62.0 us)
      constexpr int kOut = L::kGroups == 2 ? 8 : RT % 16 == 0 ? 16 : RT;
#pragma unroll 1
      for (int r = c0; r < c0 + RT && r < live; r += kOut) {
        float hi[kOut / 8][8], lo[kOut / 8][8];
#pragma unroll
        for (int c = 0; c < kOut / 8; ++c) {
          tc_load8(hi[c], lanes + kNP + r + c * 8);
          tc_load8(lo[c], lanes + 2 * kNP + r + c * 8);
        }
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < kOut; ++e)
          if (r + e < live && has_d) {
            const float o = fmaf(lo[e / 8][e % 8], 1.f / kRest, hi[e / 8][e % 8]) * sh.f[r + e];
            if (whole)
              out[int64_t(head[r + e]) * D] = __float2bfloat16_rn(o);
            else
              part[(r + e) * D] = o;
          }
      }
      tc_before();
      go = softmax_all<L::kSoft>(more && !*dead);          // all has been read before the next job writes
      if (tid == 0) mbar_arrive(&sh.job_empty[js]);
    }
  }
  __syncthreads();
  if (__builtin_expect(*dead, 0)) {
    if (tid == 0 && a.status) {
      int b = sh.start_b;
      for (long long at = sh.start_at, left = sh.share; left > 0; ++b, at = 0) {
        const long long units = sequence<R>(a, b).units;
        if (units > 0) atomicOr(a.status + b, SPEC_ST_TIMEOUT);
        left -= units - at;
      }
    }
    if (warp == kMmaWarp && lane == 0) {                   // (the thread that issued the products)
      tc_commit(&sh.drained);
      mbar_drain(&sh.drained, 0);
    }
    __syncwarp();
  }
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::kColumns));
  }
}

// Joins the partial outputs of the items that blocks share, from launch block (x, y).  Of the item that starts in block x
// and ends in a later one, each warp takes a row; where its partials are many, the launch blocks of all of its n blocks
// share the rows, and the warps of a launch block the partials of a row.
template <int R, int D>
__global__ void __launch_bounds__(32 * kMergeRows) merge_kernel(const AttnArgs a) {
  constexpr int kWide = D / 32, kMany = 8, kFlight = 4;
  __shared__ float sums[kMergeRows][D + 2];
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  wait_for_launches_before();
  let_next_start();
  SharedItem items[2];
#pragma unroll
  for (int role = 0; role < 2; ++role) items[role] = a.shared[role * kMaxGrid + blockIdx.x];
#pragma unroll
  for (int role = 0; role < 2; ++role) {
    const SharedItem& g = items[role];
    const int n = g.blocks;
    const bool many = n > kMany;
    if (n == 0 || (role == 1 && !many)) continue;
    const int worker = (int(blockIdx.x) - g.first) * int(gridDim.y) + int(blockIdx.y);
    const int step = many ? n * int(gridDim.y) : int(gridDim.y) * kMergeRows;
    for (int r = many ? worker : worker * kMergeRows + warp; r < g.live; r += step) {
      // partial k is block first's second one (k = 0) or block first + k's first
      auto slot = [&](int k) { return int64_t(2 * (g.first + k) + (k == 0)) * R + r; };
      const int k0 = many ? warp : 0, dk = many ? kMergeRows : 1;
      float x[kWide] = {}, all = 0.f, top = -INFINITY;
      for (int b = k0; b < n; b += dk * kFlight) {           // kFlight partials in flight, rescaled as they come
        float2 ml[kFlight];
        float v[kFlight][kWide];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int k = b + i * dk;
          ml[i] = make_float2(-INFINITY, 0.f);
          if (k < n) {
            ml[i] = a.part_ml[slot(k)];
            const float* p = a.part + slot(k) * D + lane * kWide;
            if constexpr (kWide == 4) {
              const float4 q = *reinterpret_cast<const float4*>(p);
              v[i][0] = q.x, v[i][1] = q.y, v[i][2] = q.z, v[i][3] = q.w;
            } else {
              const float2 q = *reinterpret_cast<const float2*>(p);
              v[i][0] = q.x, v[i][1] = q.y;
            }
          }
        }
        float rise = top;
#pragma unroll
        for (int i = 0; i < kFlight; ++i) rise = fmaxf(rise, ml[i].x);
        const float keep = all == 0.f ? 0.f : exp2f(top - rise);
        top = rise;
        all *= keep;
#pragma unroll
        for (int e = 0; e < kWide; ++e) x[e] *= keep;
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
          if (b + i * dk < n) {
            const float f = ml[i].y == 0.f ? 0.f : exp2f(ml[i].x - top);
            all += ml[i].y * f;
#pragma unroll
            for (int e = 0; e < kWide; ++e) x[e] += v[i][e] * f;
          }
      }
      if (many) {
#pragma unroll
        for (int e = 0; e < kWide; ++e) sums[warp][lane * kWide + e] = x[e];
        if (lane == 0) sums[warp][D] = all, sums[warp][D + 1] = top;
        __syncthreads();
        if (warp == 0) {
          float best = -INFINITY;
          for (int w = 0; w < kMergeRows; ++w) best = fmaxf(best, sums[w][D + 1]);
          all = 0.f;
#pragma unroll
          for (int e = 0; e < kWide; ++e) x[e] = 0.f;
          for (int w = 0; w < kMergeRows; ++w) {
            const float f = sums[w][D] == 0.f ? 0.f : exp2f(sums[w][D + 1] - best);
            all += sums[w][D] * f;
#pragma unroll
            for (int e = 0; e < kWide; ++e) x[e] += sums[w][lane * kWide + e] * f;
          }
        }
        __syncthreads();
        if (warp != 0) continue;
      }
      const float unit = all == 0.f ? 0.f : 1.f / all;
      const int row = g.row0 + r, i = row / a.group;
      const int64_t at = (int64_t(g.b) * (a.gmax + a.root) + i) * a.heads * a.group + g.h * a.group + row % a.group;
#pragma unroll
      for (int e = 0; e < kWide; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(a.out + at * D + lane * kWide + e) = __floats2bfloat162_rn(x[e] * unit, x[e + 1] * unit);
    }
  }
}

// Rows a row block takes: the rows of a kv head in as few blocks of at most 64 as hold them (each block reads the keys and
// values again), a multiple of 8 each, of 16 above 32 (two warpgroups).
int block_rows(int rows) {
  const int blocks = (rows + 63) / 64;
  const int each = (rows + blocks - 1) / blocks;
  return each > 32 ? (each + 15) / 16 * 16 : (each + 7) / 8 * 8;
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encode_map(CUtensorMap& map, const Cache& c, int which) {
  static std::atomic<Encode> known{nullptr};
  Encode encode = known.load(std::memory_order_acquire);
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return cuda_fail(e, "cuTensorMapEncodeTiled");
    if (!fn || found != cudaDriverEntryPointSuccess) {
      set_error("the driver has no cuTensorMapEncodeTiled");
      return SPEC_ECUDA;
    }
    encode = reinterpret_cast<Encode>(fn);
    known.store(encode, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {cuuint64_t(c.D), cuuint64_t(c.pages) * c.heads * c.page};
  const cuuint64_t strides[1] = {cuuint64_t(c.D)};
  const cuuint32_t box[2] = {cuuint32_t(c.D), cuuint32_t(c.page)}, ones[2] = {1, 1};
  const CUresult r = encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.codes[which], dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed with %d", int(r));
    return SPEC_ECUDA;
  }
  return SPEC_OK;
}

template <int R, int D>
int launch_attention(AttnArgs a, const Cache& c, void* ws, cudaStream_t stream) {
  using L = Layout<R, D>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const int grid = 2 * sms < kMaxGrid ? 2 * sms : kMaxGrid;
  CUtensorMap mk, mv;
  if (int rc = encode_map(mk, c, 0)) return rc;
  if (int rc = encode_map(mv, c, 1)) return rc;
  char* w = static_cast<char*>(ws);
  a.shared = reinterpret_cast<SharedItem*>(w);
  w += sizeof(SharedItem) * 2 * kMaxGrid;
  a.part_ml = reinterpret_cast<float2*>(w);
  w += sizeof(float2) * 2 * kMaxGrid * R;
  a.part = reinterpret_cast<float*>(w);
  e = cudaFuncSetAttribute(attention_kernel<R, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return cuda_fail(e, "attention shared memory");
  if (int rc = launch_early("attention kernel launch", attention_kernel<R, D>, dim3(unsigned(grid)), dim3(L::kThreads), L::kBytes, stream,
                            a, mk, mv))
    return rc;
  return launch_early("attention merge launch", merge_kernel<R, D>, dim3(unsigned(grid), unsigned((R + kMergeRows - 1) / kMergeRows)),
                      dim3(32 * kMergeRows), 0, stream, a);
}

template <int D>
int dispatch_rows(int R, const AttnArgs& a, const Cache& c, void* ws, cudaStream_t stream) {
  switch (R) {
    case 8: return launch_attention<8, D>(a, c, ws, stream);
    case 16: return launch_attention<16, D>(a, c, ws, stream);
    case 24: return launch_attention<24, D>(a, c, ws, stream);
    case 32: return launch_attention<32, D>(a, c, ws, stream);
    case 48: return launch_attention<48, D>(a, c, ws, stream);
    default: return launch_attention<64, D>(a, c, ws, stream);
  }
}

}  // namespace
}  // namespace specverify

using namespace specverify;

extern "C" size_t spec_attention_workspace_bytes(int B, int gmax, int Hq, int Hkv, int D) {
  if (B < 0 || gmax < 0 || gmax > SPEC_MAX_TREE_NODES || Hkv < 1 || Hkv > 1024 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 1024 ||
      (D != 64 && D != 128))
    return 0;
  const size_t R = size_t(block_rows((gmax + 1) * (Hq / Hkv)));
  return sizeof(SharedItem) * 2 * kMaxGrid + 2 * kMaxGrid * R * (sizeof(float2) + sizeof(float) * size_t(D));
}

extern "C" int spec_verify_attention(const spec_kv_cache_t* cache, const void* q, int dtype, const int64_t* strides, int B,
                                     int gmax, int with_root, int Hq, const int32_t* page_table, int max_pages,
                                     const int32_t* kv_len, const int32_t* num_draft, const int32_t* node_parents,
                                     float scale, void* out, int32_t* status, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  clear_error();
  if (dtype != SPEC_BF16) {
    set_error(dtype == SPEC_F32 ? "attention takes bf16 queries" : "unknown dtype code %d", dtype);
    return SPEC_EDTYPE;
  }
  if (B < 0 || gmax < 0) {
    set_error("bad sizes B=%d gmax=%d", B, gmax);
    return SPEC_EINVAL;
  }
  if (gmax > SPEC_MAX_TREE_NODES) {
    set_error("gmax=%d exceeds SPEC_MAX_TREE_NODES=%d", gmax, SPEC_MAX_TREE_NODES);
    return SPEC_ENOSPACE;
  }
  Cache c;
  if (int rc = check_cache(cache, c)) return rc;
  if (Hq < 1 || Hq % c.heads || Hq / c.heads > 1024) {
    set_error("Hq=%d is not a multiple of kv_heads=%d (up to 1024 times)", Hq, c.heads);
    return SPEC_EINVAL;
  }
  if (!std::isfinite(scale)) {
    set_error("scale is not finite");
    return SPEC_EINVAL;
  }
  const int rows = gmax + (with_root ? 1 : 0);
  if (B == 0 || rows == 0) return SPEC_OK;   // nothing to do: pointers may be null
  if (int rc = check_table(c, B, page_table, max_pages)) return rc;
  if (!q || !out || !kv_len || !workspace) {
    set_error("null required pointer (q, out, kv_len or workspace)");
    return SPEC_EINVAL;
  }
  if (c.pages == 0) {
    set_error("the cache has no pages");
    return SPEC_EINVAL;
  }
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 1) {
    set_error("q and out must be aligned to their element size");
    return SPEC_EINVAL;
  }
  if (reinterpret_cast<uintptr_t>(out) & 3) {
    set_error("out must be 4-byte aligned");
    return SPEC_EINVAL;
  }
  if (reinterpret_cast<uintptr_t>(workspace) & 15) {
    set_error("workspace must be 16-byte aligned");
    return SPEC_EINVAL;
  }
  const size_t need = spec_attention_workspace_bytes(B, gmax, Hq, c.heads, c.D);
  if (workspace_bytes < need) {
    set_error("workspace holds %zu bytes, %zu are needed", workspace_bytes, need);
    return SPEC_ENOSPACE;
  }
  const int R = block_rows((gmax + 1) * (Hq / c.heads));
  const int64_t items = int64_t((rows * (Hq / c.heads) + R - 1) / R) * c.heads;
  const int64_t tiles = int64_t(max_pages) * c.page / kTile + 1 + kItemCost;
  if (items * tiles > (int64_t(1) << 50) / B) {
    set_error("B=%d sequences of max_pages=%d pages and %d heads are too many tiles", B, max_pages, Hq);
    return SPEC_ENOSPACE;
  }
  AttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qb = strides ? strides[0] : int64_t(rows) * Hq * c.D;
  a.qn = strides ? strides[1] : int64_t(Hq) * c.D;
  a.qh = strides ? strides[2] : c.D;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ke = c.exps[0], a.ve = c.exps[1];
  a.table = page_table, a.kv_len = kv_len, a.num_draft = num_draft, a.parents = node_parents, a.status = status;
  a.pages = c.pages, a.max_pages = max_pages, a.page = c.page, a.heads = c.heads, a.group = Hq / c.heads;
  a.B = B, a.gmax = gmax, a.root = with_root ? 1 : 0;
  a.scale = scale * 1.4426950408889634f;
  a.q_vec = reinterpret_cast<uintptr_t>(q) % 8 == 0 && a.qb % 4 == 0 && a.qn % 4 == 0 && a.qh % 4 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c.D == 128 ? dispatch_rows<128>(R, a, c, workspace, st) : dispatch_rows<64>(R, a, c, workspace, st);
}

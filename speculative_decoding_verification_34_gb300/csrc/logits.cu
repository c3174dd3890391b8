// Penalties for repeated tokens, logit biases and grammar masks on the logits of a verification block.
//
// Row i of a block follows the committed context and the drafts on row i's path, so its counts are those of the history
// plus those of that path: with seen(v) and cnt(v) over them,
//     x = l > 0 ? l / r : l * r   where seen(v)            (repetition)
//     x = x - f * cnt(v) - p * [cnt(v) > 0]                (frequency, presence)
//     x = x + bias(v),  then -inf where the row's mask forbids v,
// in 32 bits, rounded once.
//
// Two parts.  The stream applies the masks alone to every vector of every row (what a mask forbids whole is not read, what
// is allowed whole is not touched in place); the fix goes over the marked ids (those of the history, the drafts and the
// biases: few of the vocabulary), row by row.  That keeps the stream short of registers and branches, and the arithmetic
// to the ids that need it.
//
// The stream is a kernel of its own that fills the SMs with loads, bound by HBM; rows whose length is no multiple of a
// vector are cut at 16-byte boundaries (20 sequences of 41 rows of 46044 bf16: 34 us, value by value 64).  The fix is a
// dependent launch, one block to a sequence or to some of its rows, that finds the marked ids while the stream ends: a
// bitmap of the vocabulary in shared memory, its ranks by a prefix sum, and an entry for each id (count, marks, last bias)
// at its rank; a draft's token has the set of drafts that are the same beside it, so a row's count of it is one population
// count.  What is left behind the stream is one round of reads and writes.  Rows that fit few vectors of one block are
// streamed by the fix itself: one launch.
//
// Measured (GB300): 128 sequences, 5 rows of 128256 bf16, 2048 tokens of history, 64 biases and masks: 61 us, of which the
// stream is 46 (a plain copy of its rows takes 44 at the measured copy rate); 8 sequences of 5 rows of 1024 fp32: 5.4 us.
// Before: all of it in one pass over table words beside the logits 363 us; the stream and then the marked ids by clusters
// with the table in shared memory 78 us (48 registers and 37 KB a block held the stream at 5.0 TB/s).

#include <cuda_bf16.h>

#include <cmath>

#include "common.cuh"
#include "tree.cuh"

namespace specverify {
namespace {

constexpr int kThreads = 256;         // of a stream block
constexpr int kFlight = 4;            // vectors whose loads one thread has in flight
constexpr int kAhead = 4;             // vectors that a thread of a streaming fix block loads before it looks for marked ids
constexpr int kPairs = 5;             // (marked id, row) pairs a fix thread has in flight
constexpr int kHeld = 8;              // history tokens a thread of a fix block holds between its two uses of them
constexpr int kEntries = 12288;       // marked ids of a window at most
constexpr int kWindow = 1 << 18;      // ids of a window at most: a 32 KB bitmap
constexpr int kFixBlocks = 152;       // blocks up to which the fix splits the rows of a sequence
constexpr int kPartRows = 4;          // rows that a part has at least
constexpr int64_t kOwn = 2048;        // vectors of a sequence up to which the fix streams them itself
constexpr int kIdBits = 24;           // of an id: at most 2^21
constexpr unsigned kSeen = 1u << 31, kBias = 1u << 30, kCount = kBias - 1;

struct LogitsArgs {
  const void* logits;
  void* out;
  int rows, first_row, V, window, entries;     // ids of a fix block, marked ids it has room for
  const int32_t *history, *committed_len, *prompt_len;
  int cap;
  const int32_t *draft_tokens, *num_draft, *node_parents;
  int gmax;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_ids;
  const float* bias_values;
  int nbias;
  const uint32_t* allowed;
  int words;
  int32_t* status;
  bool apart;                          // the stream is a launch before the fix
};

// The signs of x's bytes that the selector names, each over a byte of the result.
template <unsigned kSelector>
__device__ __forceinline__ unsigned signs(unsigned x) {
  unsigned r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "n"(kSelector));
  return r;
}

// Loads that leave the L2 first: what the stream reads is not read again, what it writes is, by the fix.
__device__ __forceinline__ uint64_t passing() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load_passing(const uint4* p, uint64_t policy) {
  uint4 x;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p), "l"(policy));
  return x;
}
template <class Raw>
__device__ __forceinline__ Raw load_passing(const Raw* p, uint64_t) {
  return *p;
}

// kVec values as the stream moves them, and -inf in the places that `ok` (a bit for each) leaves out.
template <class T, int kVec>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void forbid(Raw& r, unsigned ok) {
    // bit j of four to the sign of byte j, then each sign over two bytes
    const unsigned lo = (ok & 15) * 0x10204080u, hi = (ok >> 4) * 0x10204080u;
    const unsigned keep[4] = {signs<0x9988>(lo), signs<0xbbaa>(lo), signs<0x9988>(hi), signs<0xbbaa>(hi)};
#pragma unroll
    for (int k = 0; k < 4; ++k) (&r.x)[k] = ((&r.x)[k] & keep[k]) | (0xff80ff80u & ~keep[k]);
  }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  using Raw = unsigned short;
  static __device__ __forceinline__ void forbid(Raw& r, unsigned ok) { r = ok & 1 ? r : 0xff80u; }
};
template <>
struct Pack<float, 4> {
  using Raw = uint4;
  static __device__ __forceinline__ void forbid(Raw& r, unsigned ok) {
#pragma unroll
    for (int k = 0; k < 4; ++k) (&r.x)[k] = (ok >> k) & 1 ? (&r.x)[k] : 0xff800000u;
  }
};
template <>
struct Pack<float, 1> {
  using Raw = unsigned;
  static __device__ __forceinline__ void forbid(Raw& r, unsigned ok) { r = ok & 1 ? r : 0xff800000u; }
};

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void assign(float& o, float x) { o = x; }
__device__ __forceinline__ void assign(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }

// A parameter that is off for this sequence: not given, or not a number one can use.
__device__ __forceinline__ float setting(const float* p, int b, float off, bool positive) {
  const float x = p ? p[b] : off;
  return isfinite(x) && (!positive || x > 0.f) ? x : off;
}

// The stream: a block takes kThreads * kFlight vectors of one row.  kRagged: rows begin anywhere, alike in both arrays; their
// vectors are cut at 16-byte boundaries, the first and the last of a row are perhaps not whole and go value by value.
template <class T, int kVec, bool kRagged>
__global__ void __launch_bounds__(kThreads, 8) stream_kernel(const LogitsArgs a) {
  using P = Pack<T, kVec>;
  using Raw = typename P::Raw;
  constexpr unsigned kAll = (1u << kVec) - 1;
  wait_for_launches_before();
  let_next_start();                    // the fix may look for its marked ids
  const unsigned b = blockIdx.y / unsigned(a.rows), r = blockIdx.y - b * unsigned(a.rows);
  const int n = a.num_draft ? a.num_draft[b] : a.gmax;
  const T* in = static_cast<const T*>(a.logits) + int64_t(blockIdx.y) * a.V;
  T* out = static_cast<T*>(a.out) + int64_t(blockIdx.y) * a.V;
  const uint32_t* mask = a.allowed + int64_t(blockIdx.y) * a.words;
  const int shift = kRagged ? int(reinterpret_cast<uintptr_t>(out) & 15) / int(sizeof(T)) : 0;
  const int v0 = (int(blockIdx.x) * kThreads * kFlight + int(threadIdx.x)) * kVec - shift;
  const bool in_place = a.logits == a.out;
  auto whole = [&](int v) { return kRagged ? v >= 0 && v <= a.V - kVec : v < a.V; };
  unsigned ok[kFlight];
#pragma unroll
  for (int i = 0; i < kFlight; ++i) {
    const int v = v0 + i * kThreads * kVec;
    ok[i] = kAll;
    if (a.allowed && whole(v)) {
      unsigned bits = mask[v >> 5] >> (v & 31);
      if (kRagged && (v & 31) > 32 - kVec) bits |= mask[(v >> 5) + 1] << (32 - (v & 31));
      ok[i] = bits & kAll;
    }
  }
  if (int(r) + a.first_row > min(max(n, 0), a.gmax)) return;
  const uint64_t policy = passing();
  Raw x[kFlight];
#pragma unroll
  for (int i = 0; i < kFlight; ++i) {
    const int v = v0 + i * kThreads * kVec;
    x[i] = Raw{};
    if (whole(v) && ok[i] != 0 && !(in_place && ok[i] == kAll)) x[i] = load_passing(reinterpret_cast<const Raw*>(in + v), policy);
  }
#pragma unroll
  for (int i = 0; i < kFlight; ++i) {
    const int v = v0 + i * kThreads * kVec;
    if (whole(v) && !(in_place && ok[i] == kAll)) {
      if (a.allowed) P::forbid(x[i], ok[i]);
      *reinterpret_cast<Raw*>(out + v) = x[i];
    }
    if (kRagged && v < a.V && !whole(v)) {
#pragma unroll 1
      for (int u = max(v, 0); u < min(v + kVec, a.V); ++u) {
        T y = in[u];
        if (a.allowed && !((mask[u >> 5] >> (u & 31)) & 1)) assign(y, -INFINITY);
        out[u] = y;
      }
    }
  }
}

constexpr size_t fix_bytes(int window, int entries) { return size_t(window) / 32 * 6 + size_t(entries) * 12; }

// kStream: the block streams its sequence's rows too; else the launch before has.
template <class T, int kVec, bool kStream, int kFix>
__global__ void __launch_bounds__(kFix, 1024 / kFix) fix_kernel(const LogitsArgs a) {
  constexpr int kFixWarps = kFix / 32;
  using P = Pack<T, kVec>;
  using Raw = typename P::Raw;
  extern __shared__ unsigned shared[];
  __shared__ unsigned long long path[64];
  __shared__ unsigned long long same[64];                // drafts of draft j's token, a bit each
  __shared__ int up[64];
  __shared__ int sums[kFixWarps];
  const int words = a.window / 32;
  unsigned* const entry = shared;                        // [a.entries] marks and count of the id of that rank
  int* const ids = reinterpret_cast<int*>(entry + a.entries);     // and 1 + its first draft, above kIdBits
  int* const bias_at = ids + a.entries;                  // 1 + the last bias of an id
  unsigned* const bits = reinterpret_cast<unsigned*>(bias_at + a.entries);     // [words]
  unsigned short* const before = reinterpret_cast<unsigned short*>(bits + words);     // [words] marked ids in the words before
  // the sequences streamed last come first: their rows are still in the L2
  const int b = int(gridDim.y - 1 - blockIdx.y), tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int base = int(blockIdx.x) * a.window, limit = min(a.window, a.V - base);

  // what it reads before the wait was there before the stream's launch began
  const bool behind = !kStream && a.apart;
  if (!behind) {
    wait_for_launches_before();
    let_next_start();
  }
  // (all of these loads are independent of one another: one round trip)
  int n = a.num_draft ? a.num_draft[b] : a.gmax;
  const int committed = a.history ? a.committed_len[b] : 0, prompt = a.prompt_len ? a.prompt_len[b] : 0;
  const float rep = setting(a.repetition, b, 1.f, true);
  const float freq = setting(a.frequency, b, 0.f, false);
  const float pres = setting(a.presence, b, 0.f, false);
  const int32_t* h = a.history + int64_t(b) * a.cap;
  const int32_t* bid = a.bias_ids + int64_t(b) * a.nbias;
  auto here = [&](int id) { return unsigned(id) - unsigned(base); };       // an id's place in the window; `limit` or more: not in it
  unsigned held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = a.history && tid + k * kFix < a.cap ? here(h[tid + k * kFix]) : ~0u;
  int draft = tid < a.gmax ? a.draft_tokens[int64_t(b) * a.gmax + tid] : -1;

  const int draft_lo = warp == 1 && lane < a.gmax ? a.draft_tokens[int64_t(b) * a.gmax + lane] : -1;

  const bool clamped = n < 0 || n > a.gmax;
  n = min(max(n, 0), a.gmax);
  // this block's rows of the sequence: [first, first + rows)
  const int whole = max(min(a.rows, n + 1 - a.first_row), 0);
  const int first = kStream ? 0 : whole * int(blockIdx.z) / int(gridDim.z);
  const int rows = kStream ? whole : whole * (int(blockIdx.z) + 1) / int(gridDim.z) - first;
  const bool counts = (rep != 1.f || freq != 0.f || pres != 0.f) && rows > 0;
  const int nbias = rows > 0 ? a.nbias : 0;
  const int clen = counts && a.history ? min(max(committed, 0), a.cap) : 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (tid + k * kFix >= clen) held[k] = ~0u;
  if (tid >= n) draft = -1;

  const int64_t row0 = int64_t(b) * a.rows + first;
  const T* in = static_cast<const T*>(a.logits) + row0 * a.V;              // the sequence's rows: fewer than 2^27 values
  T* out = static_cast<T*>(a.out) + row0 * a.V;
  const uint32_t* mask = a.allowed + row0 * a.words;
  // the rows to stream: vector i is vector i % vectors of row i / vectors
  constexpr unsigned kAll = (1u << kVec) - 1;
  const bool in_place = a.logits == a.out;
  const int vectors = (limit + kVec - 1) / kVec, streamed = kStream && (a.allowed || !in_place) ? rows * vectors : 0;
  auto load = [&](int i, Raw& x, unsigned& ok, int& place) {
    place = -1;
    if (i >= streamed) return;
    const int r = i / vectors, v = base + (i - r * vectors) * kVec;
    ok = a.allowed ? (mask[r * a.words + (v >> 5)] >> (v & 31)) & kAll : kAll;
    if (in_place && ok == kAll) return;
    place = r * a.V + v;
    x = Raw{};
    if (ok != 0) x = *reinterpret_cast<const Raw*>(in + place);
  };
  auto store = [&](Raw& x, unsigned ok, int place) {
    if (place < 0) return;
    if (a.allowed) P::forbid(x, ok);
    *reinterpret_cast<Raw*>(out + place) = x;
  };
  Raw ahead[kAhead];
  unsigned ahead_ok[kAhead];
  int ahead_at[kAhead];
  if constexpr (kStream) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(tid + k * kFix, ahead[k], ahead_ok[k], ahead_at[k]);
  }

  for (int i = tid; i < words; i += kFix) bits[i] = 0;
  for (int i = tid; i < a.entries; i += kFix) entry[i] = 0, bias_at[i] = 0;
  if (warp == 1) {                     // (a thread of it holds draft lane + 32)
    unsigned long long lo = 0, hi = 0;
    for (int j = 0; j < n; ++j) {
      const int d = __shfl_sync(~0u, j < 32 ? draft_lo : draft, j & 31);
      lo |= (unsigned long long)(d == draft_lo) << j;
      hi |= (unsigned long long)(d == draft) << j;
    }
    same[lane] = lo;
    same[lane + 32] = hi;
  }
  if (warp == 0) {
    const bool bad_tree = path_masks(a.node_parents ? a.node_parents + int64_t(b) * a.gmax : nullptr, n, path, up);
    const int status = (clamped ? SPEC_ST_CLAMPED_GAMMA : 0) | (bad_tree ? SPEC_ST_BAD_TREE : 0);
    if (blockIdx.x == 0 && blockIdx.z == 0 && lane == 0 && a.status && status) atomicOr(a.status + b, status);
  }
  __syncthreads();

  // which ids are marked
  auto mark = [&](unsigned v) {
    if (v < unsigned(limit)) atomicOr(bits + (v >> 5), 1u << (v & 31));
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) mark(held[k]);
  for (int t = tid + kHeld * kFix; t < clen; t += kFix) mark(here(h[t]));
  if (counts && tid < n) mark(here(draft));
  for (int t = tid; t < nbias; t += kFix) mark(here(bid[t]));
  __syncthreads();

  // their ranks: a thread takes `each` words
  const int each = (words + kFix - 1) / kFix, w0 = min(tid * each, words), w1 = min(w0 + each, words);
  int mine = 0;
  for (int i = w0; i < w1; ++i) mine += __popc(bits[i]);
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += t;
  }
  if (lane == 31) sums[warp] = sum;
  __syncthreads();
  int at = sum - mine, total = 0;
  for (int w = 0; w < kFixWarps; ++w) {
    if (w < warp) at += sums[w];
    total += sums[w];
  }
  for (int i = w0; i < w1; ++i) {
    before[i] = (unsigned short)(at);
    at += __popc(bits[i]);
  }
  __syncthreads();

  // an entry for each, which whoever marked the id finds
  auto rank = [&](unsigned v) {
    const int r = int(before[v >> 5]) + __popc(bits[v >> 5] & ((1u << (v & 31)) - 1));
    ids[r] = base + int(v);
    return r;
  };
  auto count = [&](unsigned v, int t) {
    if (v >= unsigned(limit)) return;
    if (t < prompt)
      atomicOr(entry + rank(v), kSeen);
    else
      atomicAdd(entry + rank(v), 1u);
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) count(held[k], tid + k * kFix);
  for (int t = tid + kHeld * kFix; t < clen; t += kFix) count(here(h[t]), t);
  // the first draft of a token: its rank
  const int drafted = counts && tid < n && here(draft) < unsigned(limit) && __ffsll(same[tid]) == tid + 1 ? rank(here(draft)) : -1;
  for (int t = tid; t < nbias; t += kFix) {
    const unsigned v = here(bid[t]);
    if (v < unsigned(limit)) {
      const int r = rank(v);
      atomicOr(entry + r, kBias);
      atomicMax(bias_at + r, t + 1);
    }
  }
  __syncthreads();
  if (drafted >= 0) ids[drafted] |= (tid + 1) << kIdBits;

  if constexpr (kStream) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) store(ahead[k], ahead_ok[k], ahead_at[k]);
    for (int i = tid + kAhead * kFix; i < streamed; i += kFix) {
      Raw x;
      unsigned ok = 0;
      int place;
      load(i, x, ok, place);
      store(x, ok, place);
    }
  } else {
    if (behind) {                      // the rows are streamed
      wait_for_launches_before();
      let_next_start();
    }
  }
  __syncthreads();

  // every marked id in every row, in place; neighbouring threads take neighbouring ids
  const int pairs = total * rows;
  for (int k0 = tid; k0 < pairs; k0 += kFix * kPairs) {
    int e[kPairs], r[kPairs], place[kPairs];
    float l[kPairs];
    bool ok[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {                   // the loads of all of a thread's pairs are in flight together
      const int k = min(k0 + i * kFix, pairs - 1);
      r[i] = k / total;
      e[i] = k - r[i] * total;
      const int id = ids[e[i]] & ((1 << kIdBits) - 1);
      place[i] = r[i] * a.V + id;
      ok[i] = k0 + i * kFix < pairs;
      l[i] = value((kStream ? in : out)[place[i]]);      // (a launch before has copied it, to where the L2 may still have it)
      if (a.allowed) ok[i] = ok[i] && (mask[r[i] * a.words + (id >> 5)] >> (id & 31)) & 1;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if (!ok[i]) continue;
      const unsigned w = entry[e[i]];
      float x = l[i];
      int cnt = int(w & kCount);
      const int j = ids[e[i]] >> kIdBits;
      if (j > 0) cnt += __popcll(path[a.first_row + first + r[i]] & same[j - 1]);
      if (cnt > 0 || (w & kSeen)) x = x > 0.f ? x / rep : x * rep;
      if (cnt > 0) x = x - freq * float(cnt) - pres;
      if (w & kBias) x += a.bias_values[int64_t(b) * a.nbias + bias_at[e[i]] - 1];      // the last entry of an id counts
      assign(out[place[i]], x);
    }
  }
}

// Sequences b0 onward.
LogitsArgs shifted(const LogitsArgs& a, int b0, size_t esz) {
  LogitsArgs s = a;
  const int64_t o = b0;
  s.logits = static_cast<const char*>(a.logits) + o * a.rows * a.V * int64_t(esz);
  s.out = static_cast<char*>(a.out) + o * a.rows * a.V * int64_t(esz);
  if (a.history) s.history = a.history + o * a.cap, s.committed_len = a.committed_len + o;
  if (a.prompt_len) s.prompt_len = a.prompt_len + o;
  if (a.draft_tokens) s.draft_tokens = a.draft_tokens + o * a.gmax;
  if (a.num_draft) s.num_draft = a.num_draft + o;
  if (a.node_parents) s.node_parents = a.node_parents + o * a.gmax;
  if (a.repetition) s.repetition = a.repetition + o;
  if (a.frequency) s.frequency = a.frequency + o;
  if (a.presence) s.presence = a.presence + o;
  if (a.nbias) s.bias_ids = a.bias_ids + o * a.nbias, s.bias_values = a.bias_values + o * a.nbias;
  if (a.allowed) s.allowed = a.allowed + o * a.rows * a.words;
  if (a.status) s.status = a.status + o;
  return s;
}

template <class T, int kVec, bool kStream, int kFix>
int launch_fix(const LogitsArgs& a, const dim3& grid, cudaStream_t stream) {
  const size_t smem = fix_bytes(a.window, a.entries);
  // (the most that any call needs: the limit is the kernel's, for all threads that launch it)
  const cudaError_t e = cudaFuncSetAttribute(fix_kernel<T, kVec, kStream, kFix>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(fix_bytes(kWindow, kEntries)));
  if (e != cudaSuccess) return cuda_fail(e, "logits fix shared memory");
  return launch_early("logits fix kernel launch", fix_kernel<T, kVec, kStream, kFix>, grid, dim3(kFix), smem, stream, a);
}

template <class T, int kVec, bool kStream>
int launch_fix(const LogitsArgs& a, int B, cudaStream_t stream) {
  const int windows = (a.V + a.window - 1) / a.window, parts = (a.rows + kPartRows - 1) / kPartRows;
  const int spare = int(kFixBlocks / (int64_t(B) * windows));
  // Few sequences' rows go to several blocks, each of which finds the marked ids for itself: 64 rows of 4222 bf16 of 28
  // sequences, 2273 tokens of history: 21 us, one block each 45.
  const dim3 grid(unsigned(windows), unsigned(B), unsigned(kStream || spare < 2 ? 1 : parts < spare ? parts : spare));
  if constexpr (kStream) {
    return launch_fix<T, kVec, true, 512>(a, grid, stream);
  } else {
    // A block of 1024 threads has an SM's registers to itself.  More than there are SMs would go in two turns: 158 sequences
    // of 9 rows of 4727 bf16 17.6 us, with half the threads 11.9; but 128 of 5 rows of 128256 62.4, with half 66.
    return spare > 0 ? launch_fix<T, kVec, false, 1024>(a, grid, stream) : launch_fix<T, kVec, false, 512>(a, grid, stream);
  }
}

template <class T, int kVec, bool kRagged>
int launch_process(const LogitsArgs& args, int B, cudaStream_t stream) {
  LogitsArgs a = args;
  const bool streams = a.allowed || a.logits != a.out;
  const bool fixes = a.repetition || a.frequency || a.presence || a.nbias > 0;
  // A window's marked ids have an entry each: as many as there are tokens and biases, or, where those are more than a block
  // has room for, as the window has ids.
  const int64_t marks = fixes ? (a.history ? int64_t(a.cap) : 0) + a.gmax + a.nbias : 0;
  const int all = (a.V + 31) / 32 * 32;
  const int room = marks <= kEntries ? kWindow : kEntries;
  a.window = all < room ? all : room;
  a.entries = int(marks < a.window ? marks : a.window);
  constexpr int kOwnVec = kRagged ? 1 : kVec;
  const bool apart = a.apart = streams && int64_t(a.rows) * a.V > kOwn * kOwnVec;
  // a grid's second dimension holds at most 65535: sequences, or rows of the stream
  const int most = apart ? 65535 / a.rows : 65535;
  for (int b0 = 0; b0 < B; b0 += most) {
    const LogitsArgs s = shifted(a, b0, sizeof(T));
    const int nb = B - b0 < most ? B - b0 : most;
    if (apart) {
      const int vectors = (a.V + (kRagged ? 2 * (kVec - 1) : kVec - 1)) / kVec;
      const dim3 grid(unsigned((vectors + kThreads * kFlight - 1) / (kThreads * kFlight)), unsigned(nb * a.rows));
      if (int rc = launch_early("logits stream kernel launch", stream_kernel<T, kVec, kRagged>, grid, dim3(kThreads), 0, stream, s)) return rc;
    }
    if (apart && !fixes && !a.status) continue;          // (the fix also reports bad trees and counts)
    if (int rc = apart || !streams ? launch_fix<T, kVec, false>(s, nb, stream) : launch_fix<T, kOwnVec, true>(s, nb, stream)) return rc;
  }
  return SPEC_OK;
}

}  // namespace
}  // namespace specverify

using namespace specverify;

extern "C" int spec_process_logits(const void* logits, void* out, int dtype, int B, int rows, int first_row, int V,
                                   const int32_t* history, const int32_t* committed_len, const int32_t* prompt_len,
                                   int cap, const int32_t* draft_tokens, const int32_t* num_draft,
                                   const int32_t* node_parents, int gmax, const float* repetition,
                                   const float* frequency, const float* presence, const int32_t* bias_ids,
                                   const float* bias_values, int nbias, const uint32_t* allowed, int mask_words,
                                   int32_t* status, void* stream) {
  clear_error();
  if (dtype != SPEC_BF16 && dtype != SPEC_F32) {
    set_error("unknown dtype code %d", dtype);
    return SPEC_EDTYPE;
  }
  if (B < 0 || gmax < 0 || V < 1 || nbias < 0 || (first_row != 0 && first_row != 1)) {
    set_error("bad sizes B=%d gmax=%d V=%d nbias=%d first_row=%d", B, gmax, V, nbias, first_row);
    return SPEC_EINVAL;
  }
  if (gmax > SPEC_MAX_TREE_NODES) {
    set_error("gmax=%d exceeds SPEC_MAX_TREE_NODES=%d", gmax, SPEC_MAX_TREE_NODES);
    return SPEC_ENOSPACE;
  }
  const int vmax = dtype == SPEC_BF16 ? 1 << 21 : 1 << 20;
  if (V > vmax) {
    set_error("V=%d exceeds %d", V, vmax);
    return SPEC_ENOSPACE;
  }
  if (rows < 0 || rows > gmax + 1 - first_row) {
    set_error("rows=%d is not in [0, gmax + 1 - first_row = %d]", rows, gmax + 1 - first_row);
    return SPEC_EINVAL;
  }
  if (B == 0 || rows == 0) return SPEC_OK;   // nothing to do: pointers may be null
  if (!logits || !out || (gmax > 0 && !draft_tokens)) {
    set_error("null required pointer (logits, out or draft_tokens)");
    return SPEC_EINVAL;
  }
  if ((history != nullptr) != (committed_len != nullptr) || (prompt_len && !history)) {
    set_error("history and committed_len must be given together, prompt_len only with them");
    return SPEC_EINVAL;
  }
  if (history && (cap < 1 || cap > (1 << 28))) {
    set_error("history capacity %d is not in [1, 2^28]", cap);
    return history && cap < 1 ? SPEC_EINVAL : SPEC_ENOSPACE;
  }
  if (nbias > 0 && (!bias_ids || !bias_values)) {
    set_error("nbias=%d needs bias_ids and bias_values", nbias);
    return SPEC_EINVAL;
  }
  if (allowed && int64_t(mask_words) * 32 < V) {
    set_error("mask_words=%d holds fewer than V=%d bits", mask_words, V);
    return SPEC_EINVAL;
  }
  if (allowed && mask_words > 1 << 20) {
    set_error("mask_words=%d exceeds 2^20", mask_words);
    return SPEC_ENOSPACE;
  }
  const size_t esz = dtype == SPEC_BF16 ? 2 : 4;
  const size_t bytes = size_t(B) * rows * V * esz;
  const uintptr_t p = reinterpret_cast<uintptr_t>(logits), q = reinterpret_cast<uintptr_t>(out);
  if (p != q && p < q + bytes && q < p + bytes) {
    set_error("logits and out overlap without being the same array");
    return SPEC_EINVAL;
  }
  if ((p | q) & (esz - 1)) {
    set_error("logits and out must be aligned to their element size");
    return SPEC_EINVAL;
  }
  LogitsArgs a{logits,       out,       rows,     first_row, V,        0,      0,           history,     committed_len,
               prompt_len,   cap,       draft_tokens, num_draft, node_parents, gmax, repetition, frequency,
               presence,     bias_ids,  bias_values, nbias,  allowed,  mask_words, status, false};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = ((p | q) & 15) == 0 && (size_t(V) * esz) % 16 == 0;
  const bool alike = ((p ^ q) & 15) == 0;      // rows begin alike in both arrays, if not at a vector's boundary
  if (dtype == SPEC_BF16)
    return vec     ? launch_process<__nv_bfloat16, 8, false>(a, B, st)
           : alike ? launch_process<__nv_bfloat16, 8, true>(a, B, st)
                   : launch_process<__nv_bfloat16, 1, false>(a, B, st);
  return vec ? launch_process<float, 4, false>(a, B, st) : alike ? launch_process<float, 4, true>(a, B, st) : launch_process<float, 1, false>(a, B, st);
}

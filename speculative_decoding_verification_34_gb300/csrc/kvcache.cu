// The paged 8-bit KV cache: keys and values quantised as they are appended, read back, and the entries of a verified
// tree's path moved to the front of their block.
//
// The tutorial's §5.1-§5.2 and the "M013" card's §06 keep a cache whose valid length is rolled back to the accepted
// prefix each round; here its entries are held.  Writing tokens into a page sets the page's exponent to the least that
// holds them (kvcache.cuh): of the written tokens alone where they start the page, else together with the exponent that
// the page's earlier tokens have, whose codes are rescaled if it grows.  So what a rejected draft leaves behind is at
// most a larger exponent of the last page, until that page is written from its start again.
//
// Measured (GB300, 8 heads of 128): 8 x 4001 tokens appended as bf16 32 us (5.0 TB/s), as fp32 44 us (6.1 TB/s), 16 x 4095
// tokens read back as bf16 63 us (5.3 TB/s), as fp32 100 us; a block of 5 tokens of 128 sequences appended 3.9 us, the
// paths of 128 trees of 63 nodes kept 6.9 us, of one tree 3.6 us.
//
// All three are bound by the bytes they move (at one block of drafts, by the launch).  One group of threads owns one
// (page, head, K or V) of the pages written, so no two groups share an exponent, and holds the values in registers
// between the maximum and the rounding: they are read once.

#include <climits>
#include <type_traits>

#include "kvcache.cuh"

namespace specverify {

int check_cache(const spec_kv_cache_t* c, Cache& out) {
  if (!c) {
    set_error("null cache");
    return SPEC_EINVAL;
  }
  if (c->num_pages < 0 || c->kv_heads < 1 || (c->head_dim != 64 && c->head_dim != 128) ||
      (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)) {
    set_error("bad cache: num_pages=%d kv_heads=%d page_size=%d (16, 32, 64 or 128) head_dim=%d (64 or 128)",
              c->num_pages, c->kv_heads, c->page_size, c->head_dim);
    return SPEC_EINVAL;
  }
  if (c->kv_heads > 1024) {
    set_error("kv_heads=%d exceeds 1024", c->kv_heads);
    return SPEC_ENOSPACE;
  }
  if (int64_t(c->num_pages) * c->kv_heads * c->page_size > INT32_MAX) {
    set_error("num_pages * kv_heads * page_size exceeds 2^31 - 1");
    return SPEC_ENOSPACE;
  }
  if (c->num_pages > 0 && (!c->k_codes || !c->v_codes || !c->k_exp || !c->v_exp)) {
    set_error("null cache array");
    return SPEC_EINVAL;
  }
  if ((reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes)) & 15) {
    set_error("cache codes must be 16-byte aligned");
    return SPEC_EINVAL;
  }
  out = Cache{{c->k_codes, c->v_codes}, {c->k_exp, c->v_exp}, c->num_pages, c->kv_heads, c->page_size, c->head_dim};
  return SPEC_OK;
}

int check_table(const Cache& c, int B, const int32_t* page_table, int max_pages) {
  if (max_pages < 1 || !page_table) {
    set_error("page_table must be given with max_pages >= 1 (got %d)", max_pages);
    return SPEC_EINVAL;
  }
  if (int64_t(max_pages) * c.page > INT32_MAX - 4096) {
    set_error("max_pages=%d pages of %d tokens exceed 2^31 positions", max_pages, c.page);
    return SPEC_ENOSPACE;
  }
  return SPEC_OK;
}

namespace {

constexpr int kVec = 8;                // values a thread takes at once
constexpr int kMaxY = 65535;

struct Strides {
  int64_t b, n, h;
};

struct AppendArgs {
  Cache c;
  const void* x[2];                    // new K, V
  Strides s[2];
  int n;
  const int32_t* table;
  int max_pages;
  const int32_t *first, *count;        // position of the first new token, how many
  int32_t* status;
  int span;                            // pages that n tokens may touch
};

__device__ __forceinline__ void flag(int32_t* status, int b, int bits) {
  if (status && bits) atomicOr(status + b, bits);
}

template <class T>
struct Values;
template <>
struct Values<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const void* p) { r = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ float get(int e) const {
    const unsigned w = (&r.x)[e >> 1];
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Values<float> {
  uint4 r[2];
  __device__ __forceinline__ void load(const void* p) {
    r[0] = static_cast<const uint4*>(p)[0];
    r[1] = static_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float((&r[e >> 2].x)[e & 3]); }
};

// The largest x of a group of kGroup threads (a warp, or the whole block), in every one of them.
template <int kGroup>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
  if constexpr (kGroup > 32) {
    __shared__ float part[kGroup / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < kGroup / 32; ++w) x = fmaxf(x, part[w]);
  }
  return x;
}

// Codes of the page's tokens before slot `keep` move from exponent old to e.
template <int kGroup>
__device__ __forceinline__ void rescale(uint8_t* codes, int keep, int D, int old, int e, int lane) {
  const float f = pow2(old - e);
  for (int i = lane; i < keep * D / 16; i += kGroup) {
    uint4 q = reinterpret_cast<uint4*>(codes)[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) (&q.x)[k] = rescale_e4m3x4((&q.x)[k], f);
    reinterpret_cast<uint4*>(codes)[i] = q;
  }
}

// kGroup threads to a page, each holding kHold vectors of it.
template <class T, int kGroup, int kHold>
__global__ void __launch_bounds__(kGroup > 32 ? kGroup : 128) append_kernel(const AppendArgs a) {
  constexpr int kThreads = kGroup > 32 ? kGroup : 128;
  const Cache& c = a.c;
  const int b = int(blockIdx.y), lane = int(threadIdx.x) % kGroup;
  const int item = int(blockIdx.x) * (kThreads / kGroup) + int(threadIdx.x) / kGroup;
  if (item >= a.span * c.heads * 2) return;
  const int which = item & 1, h = int(unsigned(item >> 1) % unsigned(c.heads)), j = int(unsigned(item >> 1) / unsigned(c.heads));

  wait_for_launches_before();
  let_next_start();
  const int first = a.first[b];
  int cnt = a.count ? a.count[b] : a.n;
  const bool clamped = cnt < 0 || cnt > a.n;
  cnt = min(max(cnt, 0), a.n);
  const bool lead = item == 0 && lane == 0;
  if (lead) flag(a.status, b, (clamped ? SPEC_ST_CLAMPED_GAMMA : 0) | (first < 0 && cnt > 0 ? SPEC_ST_BAD_PAGE : 0));
  if (first < 0) return;
  const int64_t pg = int64_t(unsigned(first) / unsigned(c.page)) + j;
  const int64_t p0 = pg * c.page;                                        // the page's first position
  const int s0 = int(max(int64_t(first) - p0, int64_t(0)));              // slots written: [s0, s1)
  const int s1 = int(min(int64_t(first) + cnt - p0, int64_t(c.page)));
  if (s1 <= s0) return;
  const int pid = pg < a.max_pages ? a.table[int64_t(b) * a.max_pages + pg] : -1;

  // the written slots' values, kVec at a time: vector i is slot s0 + (i >> shift)
  const int shift = c.D == 128 ? 4 : 3, total = (s1 - s0) << shift;
  const T* src = static_cast<const T*>(a.x[which]) + b * a.s[which].b + h * a.s[which].h + (p0 + s0 - first) * a.s[which].n;
  Values<T> x[kHold];
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = lane + k * kGroup;
    if (i < total) x[k].load(src + (i >> shift) * a.s[which].n + (i & ((1 << shift) - 1)) * kVec);
  }
  // (the values are on their way while the page is looked up)
  if (pid < 0 || pid >= c.pages) {
    if (lane == 0) flag(a.status, b, SPEC_ST_BAD_PAGE);
    return;
  }
  const int64_t row = c.row(pid, h);
  uint8_t* codes = c.codes[which] + row * c.page * c.D;
  const int old = stored_exponent(c.exps[which][row]);
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (lane + k * kGroup < total) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float y = fabsf(x[k].get(e));
        if (y <= 3.4028235e38f)
          amax = fmaxf(amax, y);
        else
          bad = true;
      }
    }
  amax = group_max<kGroup>(amax);
  int e = page_exponent(amax);
  if (s0 > 0) {
    e = max(e, old);
    if (e != old) rescale<kGroup>(codes, s0, c.D, old, e, lane);
  }
  const float f = pow2(-e);
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = lane + k * kGroup;
    if (i < total) {
      unsigned q[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float y[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float z = x[k].get(w * 4 + t);
          y[t] = z == z ? z * f : 0.f;
        }
        q[w] = to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16;
      }
      *reinterpret_cast<uint2*>(codes + int64_t(s0) * c.D + i * kVec) = make_uint2(q[0], q[1]);
    }
  }
  if (lane == 0) c.exps[which][row] = int8_t(e);
  if (bad || amax > 448.f * pow2(kExpMax)) flag(a.status, b, SPEC_ST_BAD_KV);
}

struct ReadArgs {
  Cache c;
  void* out[2];
  int n, steps;
  const int32_t* table;
  int max_pages;
  const int32_t *first, *count;
  int32_t* status;
};

// A thread makes 16-byte vectors of values, each of codes of one (token, head): kReads at a time, neighbouring threads
// neighbouring vectors, a.steps times; the next step's codes are on their way while this one's values are written.
constexpr int kReads = 4;

template <class T>
__global__ void __launch_bounds__(256) read_kernel(const ReadArgs a) {
  constexpr int kCodes = 16 / int(sizeof(T));
  using Codes = typename std::conditional<kCodes == 8, uint2, unsigned>::type;
  const Cache& c = a.c;
  const int b = int(blockIdx.y), which = int(blockIdx.z);
  const unsigned head_vectors = unsigned(c.D / kCodes), row_vectors = unsigned(c.heads) * head_vectors;
  wait_for_launches_before();
  let_next_start();
  const int first = a.first ? a.first[b] : 0;
  int cnt = a.count ? a.count[b] : a.n;
  if (blockIdx.x == 0 && which == 0 && threadIdx.x == 0)
    flag(a.status, b, (cnt < 0 || cnt > a.n ? SPEC_ST_CLAMPED_GAMMA : 0) | (first < 0 && cnt > 0 ? SPEC_ST_BAD_PAGE : 0));
  cnt = min(max(cnt, 0), a.n);
  if (first < 0) return;
  const int64_t at = int64_t(blockIdx.x) * (256 * kReads * a.steps) + threadIdx.x;
  int64_t tok = at < UINT32_MAX ? unsigned(at) / row_vectors : at / row_vectors;
  unsigned rest = unsigned(at - tok * row_vectors);
  if (tok >= cnt) return;
  const int page_shift = 31 - __clz(c.page), head_shift = 31 - __clz(int(head_vectors));
  const int32_t* const table = a.table + int64_t(b) * a.max_pages;
  uint4* const out = static_cast<uint4*>(a.out[which]) + int64_t(b) * a.n * row_vectors + at;
  int64_t page_at = -1;                // the page last looked up, and its place in the cache (-1: none)
  int pid = -1;
  Codes next[kReads];
  int next_e[kReads];                  // its page's exponent, kNone: nothing to write
  constexpr int kNone = INT_MIN;
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
      next_e[k] = kNone;
      if (tok < cnt) {
        const int64_t pos = first + tok, pg = pos >> page_shift;
        if (pg != page_at) {
          page_at = pg;
          pid = pg < a.max_pages ? table[pg] : -1;
          if (pid >= c.pages) pid = -1;
        }
        if (pid >= 0) {
          const int row = (pid * c.heads + int(rest >> head_shift)) * c.page + int(pos & (c.page - 1));     // fewer than 2^31
          next_e[k] = c.exps[which][row >> page_shift];
          next[k] = *reinterpret_cast<const Codes*>(c.codes[which] + int64_t(row) * c.D + (rest & (head_vectors - 1)) * kCodes);
        } else if (rest == 0) {
          flag(a.status, b, SPEC_ST_BAD_PAGE);
        }
      }
      rest += 256;
      while (rest >= row_vectors) rest -= row_vectors, ++tok;
    }
  };
  fetch();
#pragma unroll 1
  for (int s = 0; s < a.steps; ++s) {
    Codes q[kReads];
    int e[kReads];
#pragma unroll
    for (int k = 0; k < kReads; ++k) q[k] = next[k], e[k] = next_e[k];
    if (s + 1 < a.steps) fetch();
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
      if (e[k] == kNone) continue;
      const float f = pow2(stored_exponent(int8_t(e[k])));
      uint4 o;
#pragma unroll
      for (int w = 0; w < kCodes / 4; ++w) {
        const unsigned four = reinterpret_cast<const unsigned*>(&q[k])[w];
        const float2 u = from_e4m3x2(four & 0xffffu), v = from_e4m3x2(four >> 16);
        if constexpr (sizeof(T) == 4) {
          o = make_uint4(__float_as_uint(u.x * f), __float_as_uint(u.y * f), __float_as_uint(v.x * f), __float_as_uint(v.y * f));
        } else {
          const __nv_bfloat162 x = __floats2bfloat162_rn(u.x * f, u.y * f), y = __floats2bfloat162_rn(v.x * f, v.y * f);
          (&o.x)[2 * w] = *reinterpret_cast<const unsigned*>(&x);
          (&o.x)[2 * w + 1] = *reinterpret_cast<const unsigned*>(&y);
        }
      }
      __stcs(out + (s * kReads + k) * 256, o);
    }
  }
}

struct KeepArgs {
  Cache c;
  const int32_t* table;
  int max_pages;
  const int32_t *kv_len, *path, *accepted;
  int nmax, root;
  int32_t* status;
};

// One block moves one (sequence, head, K or V): the path's codes go to shared memory with their exponents, then each
// warp writes a page of them, as append_kernel does.  Sources lie at or behind their destinations and are all read
// before the first write.
__global__ void __launch_bounds__(128) keep_kernel(const KeepArgs a) {
  __shared__ __align__(16) uint8_t code[SPEC_MAX_TREE_NODES * 128];
  __shared__ int64_t from[SPEC_MAX_TREE_NODES];
  __shared__ int exps[SPEC_MAX_TREE_NODES];
  const Cache& c = a.c;
  const int b = int(blockIdx.y), tid = int(threadIdx.x), which = int(blockIdx.x) & 1, h = int(blockIdx.x) >> 1;
  wait_for_launches_before();
  let_next_start();
  int m = a.accepted[b];
  const bool clamped = m < 0 || m > a.nmax;
  m = min(max(m, 0), a.nmax);
  const int base = a.kv_len[b];
  const bool lead = blockIdx.x == 0 && tid == 0;
  if (lead && clamped) flag(a.status, b, SPEC_ST_CLAMPED_GAMMA);
  if (m == 0) return;
  const int64_t dst = int64_t(base) + a.root;           // position of the path's first entry after the call
  int bits = base < 0 ? SPEC_ST_BAD_PAGE : 0;
  if (base >= 0 && tid < m) {
    const int node = a.path[int64_t(b) * a.nmax + tid];
    const int prev = tid ? a.path[int64_t(b) * a.nmax + tid - 1] : 0;
    if (node <= prev || node > a.nmax) {
      bits = SPEC_ST_BAD_TREE;
    } else {
      const int64_t pos = dst + node - 1, pg = pos / c.page, dg = (dst + tid) / c.page;
      const int pid = pg < a.max_pages ? a.table[int64_t(b) * a.max_pages + pg] : -1;
      const int did = dg < a.max_pages ? a.table[int64_t(b) * a.max_pages + dg] : -1;
      if (pid < 0 || pid >= c.pages || did < 0 || did >= c.pages) {
        bits = SPEC_ST_BAD_PAGE;
      } else {
        const int64_t row = c.row(pid, h);
        exps[tid] = stored_exponent(c.exps[which][row]);
        from[tid] = (row * c.page + pos % c.page) * c.D;
      }
    }
  }
  if (bits && blockIdx.x == 0) flag(a.status, b, bits);
  if (__syncthreads_or(bits)) return;                   // a bad path or page: the sequence stays as it is
  const int per = c.D / 16;
  for (int i = tid; i < m * per; i += 128)
    reinterpret_cast<uint4*>(code)[i] = *reinterpret_cast<const uint4*>(c.codes[which] + from[i / per] + (i % per) * 16);
  __syncthreads();

  const int lane = tid & 31;
  const int64_t g0 = dst / c.page, g1 = (dst + m - 1) / c.page;
  for (int64_t pg = g0 + (tid >> 5); pg <= g1; pg += 4) {
    const int64_t p0 = pg * c.page;
    const int s0 = int(max(dst - p0, int64_t(0))), s1 = int(min(dst + m - p0, int64_t(c.page)));
    const int t0 = int(p0 + s0 - dst);                  // the page's first entry of the path
    const int64_t row = c.row(a.table[int64_t(b) * a.max_pages + pg], h);
    uint8_t* codes = c.codes[which] + row * c.page * c.D;
    const int old = stored_exponent(c.exps[which][row]);
    float amax = 0.f;
    for (int i = lane; i < (s1 - s0) * per; i += 32) {
      const uint4 q = reinterpret_cast<const uint4*>(code)[t0 * per + i];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned w = (&q.x)[k];
        const float2 u = from_e4m3x2(w & 0xffffu), v = from_e4m3x2(w >> 16);
        top = fmaxf(top, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y))));
      }
      amax = fmaxf(amax, top * pow2(exps[t0 + i / per]));
    }
    amax = group_max<32>(amax);
    int e = page_exponent(amax);
    if (s0 > 0) {
      e = max(e, old);
      if (e != old) rescale<32>(codes, s0, c.D, old, e, lane);
    }
    for (int i = lane; i < (s1 - s0) * per; i += 32) {
      uint4 q = reinterpret_cast<const uint4*>(code)[t0 * per + i];
      const float f = pow2(exps[t0 + i / per] - e);
#pragma unroll
      for (int k = 0; k < 4; ++k) (&q.x)[k] = rescale_e4m3x4((&q.x)[k], f);
      *reinterpret_cast<uint4*>(codes + int64_t(s0) * c.D + i * 16) = q;
    }
    __syncwarp();
    if (lane == 0) c.exps[which][row] = int8_t(e);
  }
}

template <class T, int kGroup, int kHold>
int launch_pages(const AppendArgs& a, int B, cudaStream_t stream) {
  constexpr int kThreads = kGroup > 32 ? kGroup : 128, kItems = kThreads / kGroup;
  const dim3 grid(unsigned((a.span * a.c.heads * 2 + kItems - 1) / kItems), unsigned(B));
  return launch_early("kv append kernel launch", append_kernel<T, kGroup, kHold>, grid, dim3(kThreads), 0, stream, a);
}

// A warp takes a page of at most 16 new tokens, holding up to 8 vectors a lane; a page of more gets as many threads as
// hold it with 4 vectors each (its 2048 vectors at most: 512 threads), or 8 of bf16 up to 1024 vectors, so that a page
// is read once whatever its size.  (8 x 4001 tokens of 8 heads of 128 in pages of 64: bf16 32 us with 128 threads of
// 8 vectors, 35 with 256 of 4; fp32, twice the registers, 53 and 44.)
template <class T>
int launch_append(const AppendArgs& a, int B, cudaStream_t stream) {
  const int vectors = (a.n < a.c.page ? a.n : a.c.page) * a.c.D / kVec;
  if (a.n <= 16 || vectors <= 32 * 8)
    return launch_pages<T, 32, 8>(a, B, stream);
  if (vectors <= 128 * 4)
    return launch_pages<T, 128, 4>(a, B, stream);
  if (sizeof(T) == 2 && vectors <= 128 * 8)
    return launch_pages<T, 128, sizeof(T) == 2 ? 8 : 4>(a, B, stream);
  if (vectors <= 256 * 4)
    return launch_pages<T, 256, 4>(a, B, stream);
  return launch_pages<T, 512, 4>(a, B, stream);
}

int check_out(const void* p, const char* name) {
  if (p && !(reinterpret_cast<uintptr_t>(p) & 15)) return SPEC_OK;
  set_error(p ? "%s must be 16-byte aligned" : "null required pointer (%s)", name);
  return SPEC_EINVAL;
}

}  // namespace
}  // namespace specverify

using namespace specverify;

extern "C" int spec_kv_append(const spec_kv_cache_t* cache, const void* k, const void* v, int dtype,
                              const int64_t* strides, int B, int n, const int32_t* page_table, int max_pages,
                              const int32_t* kv_len, const int32_t* num_new, int32_t* status, void* stream) {
  clear_error();
  AppendArgs a{};
  if (dtype != SPEC_BF16 && dtype != SPEC_F32) {
    set_error("unknown dtype code %d", dtype);
    return SPEC_EDTYPE;
  }
  if (B < 0 || n < 0) {
    set_error("bad sizes B=%d n=%d", B, n);
    return SPEC_EINVAL;
  }
  if (n > 1 << 24) {
    set_error("n=%d exceeds 2^24", n);
    return SPEC_ENOSPACE;
  }
  if (int rc = check_cache(cache, a.c)) return rc;
  if (B == 0 || n == 0) return SPEC_OK;   // nothing to write: pointers may be null
  if (int rc = check_table(a.c, B, page_table, max_pages)) return rc;
  if (int rc = check_out(k, "k")) return rc;
  if (int rc = check_out(v, "v")) return rc;
  if (!kv_len) {
    set_error("null required pointer (kv_len)");
    return SPEC_EINVAL;
  }
  const int per16 = dtype == SPEC_BF16 ? 8 : 4;
  for (int i = 0; i < 2; ++i) {
    a.s[i] = strides ? Strides{strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]}
                     : Strides{int64_t(n) * a.c.heads * a.c.D, int64_t(a.c.heads) * a.c.D, a.c.D};
    if (a.s[i].b % per16 || a.s[i].n % per16 || a.s[i].h % per16) {
      set_error("strides of k and v must be whole 16-byte vectors");
      return SPEC_EINVAL;
    }
  }
  a.x[0] = k, a.x[1] = v;
  a.n = n;
  a.max_pages = max_pages;
  a.span = (n + a.c.page - 2) / a.c.page + 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t items = int64_t(a.span) * a.c.heads * 2;
  if (items > INT32_MAX) {
    set_error("n=%d tokens of %d heads need too many thread blocks", n, a.c.heads);
    return SPEC_ENOSPACE;
  }
  for (int b0 = 0; b0 < B; b0 += kMaxY) {
    const int nb = B - b0 < kMaxY ? B - b0 : kMaxY;
    const size_t esz = dtype == SPEC_BF16 ? 2 : 4;
    for (int i = 0; i < 2; ++i) a.x[i] = static_cast<const char*>(i ? v : k) + int64_t(b0) * a.s[i].b * int64_t(esz);
    a.table = page_table + int64_t(b0) * max_pages;
    a.first = kv_len + b0;
    a.count = num_new ? num_new + b0 : nullptr;
    a.status = status ? status + b0 : nullptr;
    if (int rc = dtype == SPEC_BF16 ? launch_append<__nv_bfloat16>(a, nb, st) : launch_append<float>(a, nb, st)) return rc;
  }
  return SPEC_OK;
}

extern "C" int spec_kv_read(const spec_kv_cache_t* cache, const int32_t* page_table, int max_pages, const int32_t* start,
                            const int32_t* num, int B, int n, void* k_out, void* v_out, int dtype, int32_t* status,
                            void* stream) {
  clear_error();
  ReadArgs a{};
  if (dtype != SPEC_BF16 && dtype != SPEC_F32) {
    set_error("unknown dtype code %d", dtype);
    return SPEC_EDTYPE;
  }
  if (B < 0 || n < 0) {
    set_error("bad sizes B=%d n=%d", B, n);
    return SPEC_EINVAL;
  }
  if (n > 1 << 24) {
    set_error("n=%d exceeds 2^24", n);
    return SPEC_ENOSPACE;
  }
  if (int rc = check_cache(cache, a.c)) return rc;
  if (B == 0 || n == 0) return SPEC_OK;
  if (int rc = check_table(a.c, B, page_table, max_pages)) return rc;
  if (int rc = check_out(k_out, "k_out")) return rc;
  if (int rc = check_out(v_out, "v_out")) return rc;
  a.n = n;
  a.max_pages = max_pages;
  const size_t esz = dtype == SPEC_BF16 ? 2 : 4;
  const int codes = dtype == SPEC_BF16 ? 8 : 4;        // of a 16-byte vector of values
  const int64_t vectors = int64_t(n) * a.c.heads * (a.c.D / codes);
  a.steps = 1;                                          // more where there are blocks enough for all SMs all the same
  while (a.steps < 8 && vectors * B * 2 / (256 * kReads * a.steps * 2) >= 16 * 152) a.steps *= 2;
  const int64_t blocks = (vectors + 256 * kReads * a.steps - 1) / (256 * kReads * a.steps);
  if (blocks > INT32_MAX) {
    set_error("n=%d tokens of %d heads need too many thread blocks", n, a.c.heads);
    return SPEC_ENOSPACE;
  }
  for (int b0 = 0; b0 < B; b0 += kMaxY) {
    const int nb = B - b0 < kMaxY ? B - b0 : kMaxY;
    const int64_t off = int64_t(b0) * n * a.c.heads * a.c.D * int64_t(esz);
    a.out[0] = static_cast<char*>(k_out) + off;
    a.out[1] = static_cast<char*>(v_out) + off;
    a.table = page_table + int64_t(b0) * max_pages;
    a.first = start ? start + b0 : nullptr;
    a.count = num ? num + b0 : nullptr;
    a.status = status ? status + b0 : nullptr;
    const dim3 grid(unsigned(blocks), nb, 2);
    if (int rc = launch_early("kv read kernel launch", dtype == SPEC_BF16 ? read_kernel<__nv_bfloat16> : read_kernel<float>, grid,
                              dim3(256), 0, static_cast<cudaStream_t>(stream), a))
      return rc;
  }
  return SPEC_OK;
}

extern "C" int spec_kv_keep_path(const spec_kv_cache_t* cache, const int32_t* page_table, int max_pages,
                                 const int32_t* kv_len, const int32_t* path_nodes, const int32_t* num_accepted, int B,
                                 int nmax, int with_root, int32_t* status, void* stream) {
  clear_error();
  KeepArgs a{};
  if (B < 0 || nmax < 0) {
    set_error("bad sizes B=%d nmax=%d", B, nmax);
    return SPEC_EINVAL;
  }
  if (nmax > SPEC_MAX_TREE_NODES) {
    set_error("nmax=%d exceeds SPEC_MAX_TREE_NODES=%d", nmax, SPEC_MAX_TREE_NODES);
    return SPEC_ENOSPACE;
  }
  if (int rc = check_cache(cache, a.c)) return rc;
  if (B == 0 || nmax == 0) return SPEC_OK;
  if (int rc = check_table(a.c, B, page_table, max_pages)) return rc;
  if (!kv_len || !path_nodes || !num_accepted) {
    set_error("null required pointer (kv_len, path_nodes or num_accepted)");
    return SPEC_EINVAL;
  }
  a.max_pages = max_pages;
  a.nmax = nmax;
  a.root = with_root ? 1 : 0;
  for (int b0 = 0; b0 < B; b0 += kMaxY) {
    const int nb = B - b0 < kMaxY ? B - b0 : kMaxY;
    a.table = page_table + int64_t(b0) * max_pages;
    a.kv_len = kv_len + b0;
    a.path = path_nodes + int64_t(b0) * nmax;
    a.accepted = num_accepted + b0;
    a.status = status ? status + b0 : nullptr;
    if (int rc = launch_early("kv keep path kernel launch", keep_kernel, dim3(unsigned(a.c.heads) * 2, unsigned(nb)), dim3(128), 0,
                              static_cast<cudaStream_t>(stream), a))
      return rc;
  }
  return SPEC_OK;
}

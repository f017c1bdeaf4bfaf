// Operators on a vocabulary's logits (gfx950): log probabilities of given
// tokens with entropy and top alternatives, distillation from a teacher's top
// alternatives, and both gradients. include/nvfp4.h states the definitions.
//
// Mathematics. With c = scale * log2(e), a sum over columns is held as (r, s,
// e): s = sum 2^(c z - r), e = sum 2^(c z - r) (c z - r), r an integer. So
// L = ln2 (r + log2 s) and H = ln2 (log2 s - e / s), and two sums join by
// exact powers of two. r is near the largest c z met so far, so nothing
// overflows; -inf and the types' lowest values fall out as 2^-huge = 0.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "gemm_common.h"
#include "launch.h"
#include "nvfp4.h"

namespace nvfp4 {
namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2Hi = 0.693147182464599609375f;  // float32 of ln 2
constexpr float kLn2Lo = -1.90465429995776804525e-9f;  // ln 2 - kLn2Hi
constexpr float kMost = 1e8f;          // |s| beyond it: masked below, NaN above
constexpr double kLeastTail = 1e-6;    // smaller remaining teacher mass is none
// References: of a sum that has met masked logits alone, above the bound of their
// c z (-1e8 log2 e = -1.442695e8) by so much that their terms are 0; and of a
// finished sum that met nothing, below it (the lowest in a join).
constexpr float kFirstRef = -1.4426e8f;
constexpr float kNoRef = -2e8f;
constexpr float kInf = __builtin_inff();

struct Sum {
  float r, s, e;
};

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }
__device__ __forceinline__ float fma_(float a, float b, float c) { return __builtin_fmaf(a, b, c); }

// a - b for references a <= b; 2^-300 is 0.
__device__ __forceinline__ float shift_of(float a, float b) { return fmaxf(a - b, -300.0f); }

__device__ __forceinline__ Sum join(const Sum& a, const Sum& b) {
  Sum t;
  t.r = fmaxf(a.r, b.r);
  const float da = shift_of(a.r, t.r), db = shift_of(b.r, t.r);
  const float fa = exp2_hw(da), fb = exp2_hw(db);
  t.s = fa * a.s + fb * b.s;
  t.e = fa * (a.e + da * a.s) + fb * (b.e + db * b.s);
  return t;
}

// log2 of a sum's s, as a power of two and what is left of it: 6e-8 of 1, where
// the logarithm of s itself, up to 25, is 1e-6 off.
struct Log2 {
  float whole, left;
};

__device__ __forceinline__ Log2 split_log2(float s) {
  return Log2{static_cast<float>(__builtin_amdgcn_frexp_expf(s)), log2_hw(__builtin_amdgcn_frexp_mantf(s))};
}

// ln2 (r + l) for an integer r.
__device__ __forceinline__ float to_nats(float r, float l) {
  return fma_(r, kLn2Hi, fma_(r, kLn2Lo, l * kLn2Hi));
}

// ---------------------------------------------------------------------------
// Vectors of 16 bytes, the unit of every access to the logits. Rows start at
// any element; a row's vectors are counted from the 128-byte line in which it
// starts (`skip` elements before it), so that a wave reads and writes whole
// lines: over 4096 rows of 65537 bf16 logits the gradient took 241 us with
// vectors counted from the row's first element and 217 us so (206 with stores
// that pass the caches, below). The columns at a row's two ends that fill no
// vector are single threads' business.
// ---------------------------------------------------------------------------

typedef uint32_t Raw __attribute__((ext_vector_type(4)));

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static constexpr uint32_t gone = 0xFF800000u;  // -inf
  typedef Raw Loose __attribute__((aligned(4)));
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[e]);
  }
  static __device__ __forceinline__ Raw pack(const float (&x)[4]) {
    return Raw{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
               __float_as_uint(x[3])};
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int n = 8;
  static constexpr uint32_t gone = 0xFF80FF80u;
  typedef Raw Loose __attribute__((aligned(2)));
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf16_lo(r[e]);
      x[2 * e + 1] = bf16_hi(r[e]);
    }
  }
  // bf16 pairs, nearest even
  static __device__ __forceinline__ Raw pack(const float (&x)[8]) {
    Raw r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = gemm_common::f32x2_to_bf16x2(x[2 * e], x[2 * e + 1]);
    return r;
  }
};

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(uint16_t* p, float v) {
  *p = static_cast<uint16_t>(gemm_common::f32x2_to_bf16x2(v, 0.0f));
}

// How logits are read: kKeep leaves them in the caches for a second pass.
enum { kStream = 0, kKeep = 1 };

template <typename T, int kHow>
__device__ __forceinline__ Raw load_vec(const T* p) {
  typedef typename Vec<T>::Loose Loose;
  const Loose* q = reinterpret_cast<const Loose*>(p);
  return kHow == kStream ? Raw(__builtin_nontemporal_load(q)) : Raw(*q);
}

// A row of logits as vectors: vector v holds the columns from v n - skip on.
template <typename T>
struct Row {
  const T* z;
  int vocab, skip;

  static constexpr int n = Vec<T>::n;
  // Columns are counted in 64 bits: a vocabulary may have 2^30 of them.
  __device__ __forceinline__ int64_t column(int v) const { return static_cast<int64_t>(v) * n - skip; }
  __device__ __forceinline__ bool whole(int v) const { return column(v) >= 0 && column(v) + n <= vocab; }
  __device__ __forceinline__ int vectors() const { return static_cast<int>((static_cast<int64_t>(vocab) + skip + n - 1) / n); }
  // The column outside the whole vectors that this thread takes, or -1: threads
  // 0 to 7 those before them, 8 to 15 those after.
  __device__ __forceinline__ int before() const { return skip % n ? n - skip % n : 0; }
  __device__ __forceinline__ int after() const { return static_cast<int>((static_cast<int64_t>(vocab) + skip) % n); }
  __device__ __forceinline__ int edge() const {
    const int t = threadIdx.x, column = t < 8 ? t : vocab - after() + t - 8;
    return t < 16 && taker(column) == t ? column : -1;
  }
  // The thread that takes a column so, or -1.
  __device__ __forceinline__ int taker(int column) const {
    if (column < 0 || column >= vocab) return -1;
    if (column < before()) return column;
    return column >= vocab - after() ? column - (vocab - after()) + 8 : -1;
  }
};

// The row at z, its vectors counted from the line in which `like` starts.
template <typename T>
__device__ __forceinline__ Row<T> row_at(const T* z, int64_t vocab, const T* like) {
  return Row<T>{z, static_cast<int>(vocab), static_cast<int>((reinterpret_cast<uintptr_t>(like) & 127) / sizeof(T))};
}

// Vectors first + u * NT + thread, u < U; -inf for those that are not whole.
template <typename T, int NT, int U, int kHow>
__device__ __forceinline__ void load_tile(const Row<T>& row, int first, Raw (&r)[U]) {
  constexpr int n = Vec<T>::n;
  const int v = first + static_cast<int>(threadIdx.x);
  const T* p = row.z + row.column(v);
  if (row.column(first) >= 0 && row.column(first + NT * U) <= row.vocab) {
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = load_vec<T, kHow>(p + static_cast<int64_t>(u) * NT * n);
    return;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t gone = Vec<T>::gone;
    r[u] = Raw{gone, gone, gone, gone};
    if (row.whole(v + u * NT)) r[u] = load_vec<T, kHow>(p + static_cast<int64_t>(u) * NT * n);
  }
}

// How many of a wave's vectors in a tile hold anything of the vectors below
// `hi` (the same in all its lanes).
template <int NT, int U>
__device__ __forceinline__ int used_of(int first, int hi) {
  const int left = hi - first - static_cast<int>(threadIdx.x & ~63u);
  const int used = (left + NT - 1) / NT;
  return __builtin_amdgcn_readfirstlane(used < U ? used : U);
}

// The tiles of one workgroup, in vectors.
struct Range {
  int lo, hi;
};

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------

// What a row's scale gives: c = scale log2 e, and the bounds of unmasked z.
struct Scale {
  float c, low, high;
};

__device__ __forceinline__ Scale scale_of(float scale) {
  const float most = kMost / scale;
  return Scale{scale * kLog2e, -most, most};
}

// A sum in the making: logits above `next` move the reference to them.
struct Running {
  Sum t;
  float next;
};

__device__ __forceinline__ Running running(const Scale& c) {
  return Running{{kFirstRef, 0.0f, 0.0f}, c.low};
}

// max(a, b, c); a NaN may be passed over.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

template <int n>
__device__ __forceinline__ float max_of(const float (&x)[n]) {
  float m = max3(x[0], x[1], x[2]);
#pragma unroll
  for (int e = 3; e + 1 < n; e += 2) m = max3(m, x[e], x[e + 1]);
  return max3(m, x[n - 1], x[n - 1]);
}

// Adds logits, the largest of which is `top`. |c z| < 2^28, so r is off c z by
// 8 at most where it is too large for a fraction; and logits up to 8 (in log2)
// above the reference are taken as they come, which costs a sum nothing and
// leaves the entropy's e an error of 8 u. A masked logit's term is 0 by itself
// unless the reference is below kFirstRef (see without_masked).
template <bool kEntropy, int n>
__device__ __forceinline__ void add_logits(Running& a, const float (&z)[n], float top, const Scale& c) {
  if (top > a.next) {
    const float r = top > c.high ? __builtin_nanf("") : rintf(top * c.c);
    // the first unmasked logit may lie below kFirstRef: nothing has been summed then
    const float d = fminf(shift_of(a.t.r, r), 0.0f), f = exp2_hw(d);
    a.t.e = f * (a.t.e + d * a.t.s);
    a.t.s *= f;
    a.t.r = r;
    a.next = top + 8.0f / c.c;
  }
#pragma unroll
  for (int e = 0; e < n; ++e) {
    const float y = fma_(z[e], c.c, -a.t.r);
    const float p = exp2_hw(y);
    a.t.s += p;
    if (kEntropy) a.t.e = fma_(p, fmaxf(y, -300.0f), a.t.e);  // 0 * -inf must not arise
  }
}

template <bool kEntropy>
__device__ __forceinline__ void add_one(Running& a, float z, const Scale& c) {
  const float one[1] = {z <= c.low ? -kInf : z};
  add_logits<kEntropy>(a, one, one[0], c);
}

// The thread's sum over its vectors of `in` again where its reference has stayed
// below kFirstRef: all it has met lies within 7000 of the mask's bound, and
// masked logits may have counted. out(column): whether a column is left out too.
// In the pass itself the comparisons, though in a branch that is hardly ever
// taken, cost 2048 x 131072 bf16 (distillation) 86 to 93 us instead of 84.
template <typename T, int NT, bool kEntropy, typename F>
__device__ __forceinline__ void without_masked(Running& a, const Row<T>& row, const Range& in, const Scale& c, F out) {
  if (!(a.t.r < kFirstRef)) return;
  constexpr int n = Vec<T>::n;
  a = running(c);
#pragma unroll 1
  for (int v = in.lo + static_cast<int>(threadIdx.x); v < in.hi; v += NT) {
    if (!row.whole(v)) continue;
    float x[n];
    Vec<T>::unpack(load_vec<T, kKeep>(row.z + row.column(v)), x);
    // as bits first: written as `if (... || out(...)) x[e] = -kInf`, clang 22 for
    // gfx950 dropped the assignment where out() is true
    uint32_t gone = 0;
#pragma unroll
    for (int e = 0; e < n; ++e) {
      uint32_t drop = x[e] <= c.low;
      if (!drop) drop = out(row.column(v) + e);
      gone |= drop << e;
    }
#pragma unroll
    for (int e = 0; e < n; ++e) x[e] = gone >> e & 1u ? -kInf : x[e];
    add_logits<kEntropy>(a, x, max_of(x), c);
  }
}

__device__ __forceinline__ Sum finished(const Running& a) {
  return Sum{a.t.s == 0.0f ? kNoRef : a.t.r, a.t.s, a.t.e};
}

// Reductions over a wave by DPP moves (the result in every lane).
template <int kCtrl, int kRowMask>
__device__ __forceinline__ float moved(float v, float fill) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(fill), __float_as_uint(v), kCtrl,
                                                     kRowMask, 0xF, false));
}
__device__ __forceinline__ float from_last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += moved<0x111, 0xF>(v, 0.0f);  // row_shr 1, 2, 4, 8
  v += moved<0x112, 0xF>(v, 0.0f);
  v += moved<0x114, 0xF>(v, 0.0f);
  v += moved<0x118, 0xF>(v, 0.0f);
  v += moved<0x142, 0xA>(v, 0.0f);  // row_bcast 15, 31
  v += moved<0x143, 0xC>(v, 0.0f);
  return from_last_lane(v);
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, moved<0x111, 0xF>(v, v));
  v = fmaxf(v, moved<0x112, 0xF>(v, v));
  v = fmaxf(v, moved<0x114, 0xF>(v, v));
  v = fmaxf(v, moved<0x118, 0xF>(v, v));
  v = fmaxf(v, moved<0x142, 0xA>(v, v));
  v = fmaxf(v, moved<0x143, 0xC>(v, v));
  return from_last_lane(v);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Words in LDS for one reduction over NT threads.
template <int NT>
struct Shared {
  Sum sum[NT / 64];
};

__device__ __forceinline__ Sum wave_join(Sum t) {
  const float r = wave_max(t.r), d = shift_of(t.r, r), f = exp2_hw(d);
  return Sum{r, wave_sum(f * t.s), wave_sum(f * (t.e + d * t.s))};
}

// The sum over the workgroup, in every thread: every wave joins the waves' sums.
template <int NT>
__device__ __forceinline__ Sum block_join(const Sum& t, Shared<NT>& lds) {
  const Sum own = wave_join(t);
  const int lane = threadIdx.x & 63;
  __syncthreads();
  if (lane == 0) lds.sum[threadIdx.x >> 6] = own;
  __syncthreads();
  return wave_join(lane < NT / 64 ? lds.sum[lane] : Sum{kNoRef, 0.0f, 0.0f});
}

// ---------------------------------------------------------------------------
// The k largest logits of a row.
//
// The pass keeps, of each thread's vectors of a span of tiles, the largest
// logit, its vector and the largest logit of the span's other vectors, in LDS.
// After the pass the k-th largest of the threads' maxima (of 256 threads or
// groups of threads) bounds the k-th largest logit from below, k different
// logits reaching it, and hardly more do: with 64 of 131072 Gaussian logits
// about 75. Only vectors that may reach the bound are read again (a line of
// 128 bytes each), and their logits from the bound on go to a list of words
// (order of the value, falling column), sorted by counting. The pass itself has
// no barrier and no branch for all this: at 4096 x 131072 bf16 and k = 64 a
// selection tile by tile (a bar, a queue of vectors, two barriers) took 250 us,
// of which 90 were its own; reading whole spans again 221; this 199.
// Where more logits reach the bound than the list holds (many equal ones), the
// row is read again in order, a vector a thread at a time.
// ---------------------------------------------------------------------------

constexpr int kGroups = 256;  // maxima that the bound is taken from
constexpr int kRank = 256;    // words that are sorted by counting
constexpr int kSpans = 8;     // of a workgroup's tiles
constexpr int kPicked = 512;  // vectors that are read again

template <int NT>
struct Top {
  static constexpr int list_size = NT < 1024 ? 1024 : 2048;
  unsigned long long list[list_size];
  uint32_t group_max[kGroups];
  uint32_t span[kSpans][NT];  // as span_word gives it
  int picked_vector[kPicked];
  int picked, listed;
  uint32_t bound;
};

template <int kCtrl>
__device__ __forceinline__ uint32_t quad_moved(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), kCtrl, 0xF, 0xF, false));
}

// Unsigned integers in the order of the floats (-0 as +0; no NaN).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// A thread's span: in 16 bits the largest logit's order key, in 12 that of the
// largest logit of its other vectors, in 4 the largest one's vector.
__device__ __forceinline__ uint32_t span_word(float first, float second, int at) {
  return (order_key(first) & 0xFFFF0000u) | (order_key(second) >> 20 << 4) | (static_cast<uint32_t>(at) & 15u);
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
}

// A logit as a word of the list: in the order of the value, equal ones by
// falling column.
__device__ __forceinline__ unsigned long long word_of(float v, int64_t column) {
  return (static_cast<unsigned long long>(order_key(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(column));
}

// A place for each thread that has something, from a counter in LDS. The order
// among the waves does not matter: all that is placed so is sorted later, or
// only looked through.
__device__ __forceinline__ int claim(int& counter, bool has) {
  const uint64_t m = __ballot(has);
  if (m == 0) return 0;
  int base = 0;
  const int lead = __ffsll(static_cast<unsigned long long>(m)) - 1;
  if (static_cast<int>(threadIdx.x & 63) == lead) base = atomicAdd(&counter, __popcll(m));
  return __builtin_amdgcn_readlane(base, lead) + lanes_below(m);
}

// Keeps the list's words from `bound` on; their number.
template <int NT>
__device__ __forceinline__ int narrow(Top<NT>& t, int n, unsigned long long bound) {
  constexpr int each = Top<NT>::list_size / NT;
  unsigned long long own[each];
#pragma unroll
  for (int s = 0; s < each; ++s) {
    const int i = s * NT + static_cast<int>(threadIdx.x);
    own[s] = i < n ? t.list[i] : 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) t.listed = 0;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < each; ++s) {
    const bool has = own[s] >= bound && own[s] != 0;
    const int place = claim(t.listed, has);
    if (has) t.list[place] = own[s];
  }
  __syncthreads();
  return t.listed;
}

// Sorts the list's n words (all different) in falling order and keeps k. A
// long list is first cut at a bound that at least k words reach: the k-th
// largest, in its upper 16 bits, of 256 words spread over the list; where that
// leaves over kRank words (many equal logits), the k-th largest itself. Every
// wave searches for the bound by itself, a bit at a time.
template <int NT>
__device__ int keep_best(Top<NT>& t, int n, int k) {
  __syncthreads();
  const int lane = threadIdx.x & 63;
  if (n > 128 && n > k) {
    uint32_t key[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int i = s * 64 + lane;
      const int at = n <= 256 ? i : i * n >> 8;
      key[s] = at < n ? static_cast<uint32_t>(t.list[at] >> 48) : 0u;
    }
    uint32_t high = 0;
#pragma unroll 1
    for (int b = 15; b >= 0; --b) {
      const uint32_t next = high | (1u << b);
      int c = 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) c += __popcll(__ballot(key[s] >= next));
      if (c >= k) high = next;
    }
    n = narrow(t, n, static_cast<unsigned long long>(high) << 48);
    if (n > kRank) {
      unsigned long long bound = 0;
#pragma unroll 1
      for (int b = 63; b >= 0; --b) {
        const unsigned long long next = bound | (1ull << b);
        int c = 0;
        for (int s = 0; s < n; s += 64) c += __popcll(__ballot(s + lane < n && t.list[s + lane] >= next));
        if (c >= k) bound = next;
      }
      n = narrow(t, n, bound);
    }
  }
  // n <= kRank here: at most 128, at most k, or narrowed
  const int i = threadIdx.x;
  const unsigned long long own = i < n ? t.list[i] : 0;
  int place = 0;
  if ((i & ~63) < n) {
#pragma unroll 8
    for (int j = 0; j < n; ++j) place += t.list[j] > own;
  }
  __syncthreads();
  if (i < n && place < k) t.list[place] = own;
  __syncthreads();
  return n < k ? n : k;
}

// ---------------------------------------------------------------------------
// How the rows are cut: a workgroup takes `tiles` tiles of one row. With one
// workgroup a row it also finishes the row; else the parts' sums and lists go
// to the workspace and a second kernel joins them.
// ---------------------------------------------------------------------------

struct Cut {
  int parts;  // workgroups a row
  int tiles;  // tiles a workgroup
};

template <int NT, int U>
__device__ __forceinline__ Range range_of(const Cut& cut, int part, int vectors) {
  const int64_t each = static_cast<int64_t>(cut.tiles) * (NT * U), lo = part * each;
  return Range{static_cast<int>(lo < vectors ? lo : vectors),
               static_cast<int>(lo + each < vectors ? lo + each : vectors)};
}

// Whether the workgroup's tiles hold a column of the row.
template <typename T>
__device__ __forceinline__ bool holds(const Row<T>& row, const Range& in, int64_t column) {
  if (column < 0 || column >= row.vocab) return false;
  const int v = static_cast<int>((column + row.skip) / Vec<T>::n);
  return v >= in.lo && v < in.hi;
}

// Appends the words of the threads that have one; grows the count only beyond
// the list's end.
template <int NT>
__device__ __forceinline__ void append(Top<NT>& t, bool has, float x, int64_t column) {
  const int place = claim(t.listed, has);
  if (has && place < Top<NT>::list_size) t.list[place] = word_of(x, column);
}

// The row's k best from the beginning, in order: a later logit counts only
// above the k-th best so far (of equals the first wins), so a row of equal
// logits is passed over after its first vectors.
template <typename T, int NT>
__device__ int select_in_order(Top<NT>& t, const Row<T>& row, const Range& in, int edge, float x_edge,
                               const Scale& c, int k) {
  constexpr int n = Vec<T>::n;
  int held = 0;
  float bar = c.low;
  const auto room = [&]() {
    held = keep_best(t, held, k);
    if (held == k) bar = fmaxf(bar, key_value(static_cast<uint32_t>(t.list[k - 1] >> 32)));
  };
  const auto add = [&](bool has, float x, int64_t column) {
    if (held + NT > Top<NT>::list_size) room();
    __syncthreads();
    if (threadIdx.x == 0) t.listed = held;
    __syncthreads();
    append(t, has && x >= bar, x, column);
    __syncthreads();
    held = t.listed;
  };
  add(threadIdx.x < 8 && edge >= 0 && x_edge > c.low, x_edge, edge);
#pragma unroll 1
  for (int first = in.lo; first < in.hi; first += NT) {
    const int v = first + static_cast<int>(threadIdx.x);
    float x[n];
#pragma unroll
    for (int e = 0; e < n; ++e) x[e] = -kInf;
    if (v < in.hi && row.whole(v)) Vec<T>::unpack(load_vec<T, kStream>(row.z + row.column(v)), x);
    const float above = bar;
    if (!__syncthreads_or(max_of(x) > above)) continue;
#pragma unroll 1
    for (int e = 0; e < n; ++e) {
      float one = x[0];
#pragma unroll
      for (int j = 1; j < n; ++j) one = e == j ? x[j] : one;
      add(one > above, one, row.column(v) + e);
    }
  }
  add(threadIdx.x >= 8 && edge >= 0 && x_edge > c.low, x_edge, edge);
  return keep_best(t, held, k);
}

// The k best of the workgroup's tiles, sorted in the list; their number.
// all: order key of the thread's largest logit in whole vectors; edge and x_edge:
// its single column.
template <typename T, int NT, int U>
__device__ int select_best(Top<NT>& t, const Row<T>& row, const Range& in, int spans, int span_tiles, uint32_t all,
                           int edge, float x_edge, const Scale& c, int k) {
  constexpr int n = Vec<T>::n;
  constexpr int group = NT / kGroups;
  const uint32_t masked = order_key(c.low);
  if (group >= 2) all = max(all, quad_moved<0xB1>(all));  // quad_perm [1, 0, 3, 2]
  if (group >= 4) all = max(all, quad_moved<0x4E>(all));  // quad_perm [2, 3, 0, 1]
  if (threadIdx.x % group == 0) t.group_max[threadIdx.x / group] = all;
  if (threadIdx.x == 0) t.picked = t.listed = 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    // the largest bound, of the upper 16 bits, that k groups' maxima reach
    uint32_t key[kGroups / 64];
#pragma unroll
    for (int g = 0; g < kGroups / 64; ++g) key[g] = t.group_max[g * 64 + threadIdx.x] >> 16;
    uint32_t found = 0;
#pragma unroll
    for (int b = 15; b >= 0; --b) {
      const uint32_t next = found | (1u << b);
      int reach = 0;
#pragma unroll
      for (int g = 0; g < kGroups / 64; ++g) reach += __popcll(__ballot(key[g] >= next));
      if (reach >= k) found = next;
    }
    if (threadIdx.x == 0) t.bound = found;
  }
  __syncthreads();
  const uint32_t bound = t.bound;
  const int each = span_tiles * U;  // vectors of a span
  const auto take = [&](int v) {
    if (v >= in.hi || !row.whole(v)) return;
    float x[n];
    Vec<T>::unpack(load_vec<T, kKeep>(row.z + row.column(v)), x);
    uint32_t pass = 0;
#pragma unroll
    for (int e = 0; e < n; ++e) pass |= x[e] > c.low && order_key(x[e]) >> 16 >= bound ? 1u << e : 0u;
    if (!pass) return;
    int place = atomicAdd(&t.listed, __popc(pass));
#pragma unroll
    for (int e = 0; e < n; ++e)
      if (pass >> e & 1u) {
        if (place < Top<NT>::list_size) t.list[place] = word_of(x[e], row.column(v) + e);
        ++place;
      }
  };
  // f(first vector, their number), NT apart, for the thread's spans that reach
  // the bound with an unmasked logit: one vector, or all of the span
  const auto each_pick = [&](auto f) {
    for (int i = 0; i < spans; ++i) {
      const uint32_t own = t.span[i][threadIdx.x];
      if (own >> 16 < bound || own >> 16 < masked >> 16) continue;
      const bool all_of = each > 16 || (own >> 4 & 0xFFFu) >= bound >> 4;
      const int from = all_of ? 0 : static_cast<int>(own & 15u);
      f(in.lo + (i * each + from) * NT + static_cast<int>(threadIdx.x), all_of ? each : 1);
    }
  };
  each_pick([&](int v, int count) {
    const int place = atomicAdd(&t.picked, count);
    for (int q = 0; q < count && place + q < kPicked; ++q) t.picked_vector[place + q] = v + q * NT;
  });
  append(t, edge >= 0 && x_edge > c.low && order_key(x_edge) >> 16 >= bound, x_edge, edge);
  __syncthreads();
  const int picked = t.picked;
  if (picked <= kPicked) {
    for (int i = threadIdx.x; i < picked; i += NT) take(t.picked_vector[i]);
  } else {
    each_pick([&](int v, int count) {
      for (int q = 0; q < count; ++q) take(v + q * NT);
    });
  }
  __syncthreads();
  const int listed = t.listed;
  if (listed <= Top<NT>::list_size) return keep_best(t, listed, k);
  return select_in_order(t, row, in, edge, x_edge, c, k);
}

struct Part {
  float r, s, e, pad;
};

__device__ __forceinline__ Part* part_sums(const LogitsLaunch& a) { return static_cast<Part*>(a.ws); }
__device__ __forceinline__ unsigned long long* part_lists(const LogitsLaunch& a, int parts) {
  return reinterpret_cast<unsigned long long*>(part_sums(a) + a.rows * parts);
}

// ---------------------------------------------------------------------------
// Token log probabilities
// ---------------------------------------------------------------------------

// Log probability of the row's token, whose logit is x where it has one;
// l2 = log2 s of the row's sum t.
__device__ __forceinline__ float token_logp(int64_t vocab, int64_t token, float x, const Scale& c,
                                            const Sum& t, float l2, bool* bad) {
  if (token < 0) return 0.0f;
  if (token >= vocab) {
    *bad = true;
    return __builtin_nanf("");
  }
  if (t.s != t.s) return t.s;
  if (x <= c.low) return -kInf;
  return (fma_(x, c.c, -t.r) - l2) * kLn2Hi;
}

// The row's token (-1: none) and its logit, for thread 0.
template <typename T>
__device__ __forceinline__ int64_t load_token(const LogitsLaunch& a, const T* z, int64_t row, float* x) {
  *x = 0.0f;
  if (threadIdx.x != 0 || a.tokens == nullptr) return -1;
  const int64_t token = a.tokens[row];
  if (token >= 0 && token < a.vocab) *x = load_one(z + token);
  return token;
}

// Writes a row's outputs from its sum and, with alternatives, its sorted list
// of n words.
__device__ __forceinline__ void finish_logprobs(const LogitsLaunch& a, int64_t row, int64_t token, float x,
                                                const Sum& t, const unsigned long long* list, int n,
                                                const Scale& c) {
  const bool nan = t.s != t.s, empty = t.s == 0.0f;
  const float l2 = log2_hw(t.s);
  if (threadIdx.x == 0) {
    bool bad = nan;
    a.lse[row] = empty ? -kInf : to_nats(t.r, l2);
    if (a.entropy) a.entropy[row] = empty ? 0.0f : (l2 - t.e / t.s) * kLn2Hi;
    if (a.logp) a.logp[row] = token_logp(a.vocab, token, x, c, t, l2, &bad);
    if (bad && a.dev_status) *a.dev_status = 1;
  }
  const int j = threadIdx.x;
  if (j < a.k) {
    const unsigned long long word = j < n ? list[j] : 0;
    const uint32_t key = static_cast<uint32_t>(word >> 32);
    int32_t id = -1;
    float lp = nan ? t.s : -kInf;
    if (key != 0 && !nan) {
      id = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(word));
      lp = (fma_(key_value(key), c.c, -t.r) - l2) * kLn2Hi;
    }
    a.top_ids[row * a.k + j] = id;
    a.top_logp[row * a.k + j] = lp;
  }
}

template <int NT, bool kTop>
struct TopLds {};
template <int NT>
struct TopLds<NT, true> {
  Top<NT> t;
};

// One pass: sums, and of the alternatives three numbers per thread and span. A
// logit costs about nine slots of the vector unit with the entropy (four of them
// the exponential), and reading bf16 at the full rate leaves eleven: 8191 x
// 50001 bf16 with entropy takes 126 us (6.5 TB/s, the unit 0.84 busy), 4096 x
// 131072 with entropy and 64 alternatives 180 (6.0 TB/s, 0.87). One row of
// 131072 with 20 alternatives takes 15 us: the latency of one CU's loads, then
// of the selection.
template <typename T, int NT, int U, bool kTop, bool kEntropy>
__global__ __launch_bounds__(NT) void token_logprobs_kernel(LogitsLaunch a, Cut cut) {
  __shared__ Shared<NT> lds;
  __shared__ TopLds<NT, kTop> top;
  constexpr int n = Vec<T>::n;
  const int64_t at = blockIdx.x / cut.parts;
  const int part = static_cast<int>(blockIdx.x % cut.parts);
  const T* z = static_cast<const T*>(a.z) + at * a.ldz;
  const Row<T> row = row_at(z, a.vocab, z);
  const Range in = range_of<NT, U>(cut, part, row.vectors());
  const Scale c = scale_of(a.scale);
  float x_token;
  const int64_t token = load_token(a, z, at, &x_token);
  Running run = running(c);
  int edge = row.edge();
  if (!holds(row, in, edge)) edge = -1;
  const float x_edge = edge >= 0 ? load_one(z + edge) : -kInf;
  const int span_tiles = (cut.tiles + kSpans - 1) / kSpans;
  int spans = 0, tiles = 0, span_at = 0;
  float span_max = -kInf, span_next = -kInf, all_max = -kInf;
  for (int first = in.lo; first < in.hi; first += NT * U) {
    Raw r[U];
    // a few rows stay in the L2 for the vectors that are read again
    load_tile<T, NT, U, kTop && NT == 1024 ? kKeep : kStream>(row, first, r);
    const int used = used_of<NT, U>(first, in.hi);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= used) continue;
      float x[n];
      Vec<T>::unpack(r[u], x);
      const float largest = max_of(x);
      add_logits<kEntropy>(run, x, largest, c);
      if (kTop) {
        span_next = __builtin_amdgcn_fmed3f(span_max, span_next, largest);
        span_at = largest > span_max ? tiles * U + u : span_at;
        span_max = fmaxf(span_max, largest);
      }
    }
    if constexpr (kTop) {
      if (++tiles == span_tiles || first + NT * U >= in.hi) {
        top.t.span[spans++][threadIdx.x] = span_word(span_max, span_next, span_at);
        all_max = fmaxf(all_max, span_max);
        span_max = span_next = -kInf;
        tiles = 0;
      }
    }
  }
  without_masked<T, NT, kEntropy>(run, row, in, c, [](int64_t) { return false; });
  if (edge >= 0) add_one<kEntropy>(run, x_edge, c);
  int found = 0;
  const unsigned long long* list = nullptr;
  if constexpr (kTop) {
    found = select_best<T, NT, U>(top.t, row, in, spans, span_tiles, order_key(all_max), edge, x_edge, c, a.k);
    list = top.t.list;
  }
  const Sum t = block_join(finished(run), lds);
  if (cut.parts == 1) {
    finish_logprobs(a, at, token, x_token, t, list, found, c);
    return;
  }
  if (threadIdx.x == 0) part_sums(a)[blockIdx.x] = Part{t.r, t.s, t.e, 0.0f};
  const int j = threadIdx.x;
  if (kTop && j < a.k) {
    // places without a logit: small words, all different within the row
    part_lists(a, cut.parts)[static_cast<int64_t>(blockIdx.x) * a.k + j] = j < found ? list[j] : 1 + part * a.k + j;
  }
}

// The sum of a row's parts.
template <int NT>
__device__ __forceinline__ Sum join_parts(const LogitsLaunch& a, int64_t at, const Cut& cut, Shared<NT>& lds) {
  Sum t = {kNoRef, 0.0f, 0.0f};
  for (int p = threadIdx.x; p < cut.parts; p += NT) {
    const Part q = part_sums(a)[at * cut.parts + p];
    t = join(t, Sum{q.r, q.s, q.e});
  }
  return block_join(t, lds);
}

// Finishes rows that were cut into parts.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void token_logprobs_join_kernel(LogitsLaunch a, Cut cut) {
  __shared__ Shared<NT> lds;
  __shared__ Top<NT> top;
  const int64_t at = blockIdx.x;
  const Scale c = scale_of(a.scale);
  float x_token;
  const int64_t token = load_token(a, static_cast<const T*>(a.z) + at * a.ldz, at, &x_token);
  const Sum t = join_parts(a, at, cut, lds);
  int n = 0;
  const unsigned long long* lists = part_lists(a, cut.parts) + at * cut.parts * a.k;
  const int all = cut.parts * a.k;
  for (int from = 0; from < all;) {
    const int m = all - from < Top<NT>::list_size - n ? all - from : Top<NT>::list_size - n;
    for (int i = threadIdx.x; i < m; i += NT) top.list[n + i] = lists[from + i];
    from += m;
    n = keep_best(top, n + m, a.k);
  }
  finish_logprobs(a, at, token, x_token, t, top.list, n, c);
}

// ---------------------------------------------------------------------------
// Gradients. Outside a few columns of the row (its token, its label, the
// teacher's alternatives) the gradient is 2^(...) times a factor of the row.
// Those few are worked out before the pass and written over its result after
// it, so the pass itself knows nothing of them.
// ---------------------------------------------------------------------------

// Exponent c z - ref, or (scale z - ref) log2 e, which keeps what ref holds of
// a given L.
enum { kFromLse = 0, kFromRef = 1 };

struct Factor {
  float a, b;  // gradient = p (a + b (scale z - ref))
  float ref;
};

// Where p is 0 the gradient is: a is finite (rows with NaN have a pass of their
// own), and with b the product is kept from 0 * inf.
template <typename T, bool kEntropy, int kFrom>
__device__ __forceinline__ Raw gradient_of(const Raw& r, float scale, const Factor& f, const Scale& c) {
  constexpr int n = Vec<T>::n;
  float x[n];
  Vec<T>::unpack(r, x);
#pragma unroll
  for (int e = 0; e < n; ++e) {
    if (kFrom == kFromRef) {
      x[e] = exp2_hw(fma_(x[e], c.c, -f.ref)) * f.a;
    } else {
      const float lp = fma_(x[e], scale, -f.ref);
      const float p = exp2_hw(lp * kLog2e);
      x[e] = p * (kEntropy ? fma_(fmaxf(lp, -1000.0f), f.b, f.a) : f.a);
    }
  }
  return Vec<T>::pack(x);
}

// Stores a whole vector of the row to dz (the row's first column), past the
// caches: whole lines, which nothing here reads again. As ordinary stores the
// gradient of 4096 x 100003 bf16 logits took 360 us instead of 319, of 4096 x
// 65537 215 instead of 206.
template <typename T>
__device__ __forceinline__ void store_whole(T* dz, const Row<T>& row, int v, const Raw& r) {
  __builtin_nontemporal_store(r, reinterpret_cast<typename Vec<T>::Loose*>(dz + row.column(v)));
}

// A logit as the first element of a vector, and back.
__device__ __forceinline__ uint32_t as_word(uint16_t v) { return v; }
__device__ __forceinline__ uint32_t as_word(float v) { return __float_as_uint(v); }
template <typename T>
__device__ __forceinline__ T from_word(uint32_t w) {
  if constexpr (sizeof(T) == 2) return static_cast<uint16_t>(w);
  else return __uint_as_float(w);
}

// Whether masked logits may lie so near to ref that their p is not 0 by itself:
// they get it below 2^-9000 only where ref is above kFirstRef (in log2; in nats
// -9.9992e7, taken a little higher).
template <int kFrom>
__device__ __forceinline__ bool beside_masked(const Factor& f) {
  return f.ref < (kFrom == kFromRef ? kFirstRef : -0.9999e8f);
}

// The gradient of rows beside masked logits: a vector at a time, masked ones by
// themselves.
template <typename T, int NT, bool kEntropy, int kFrom>
__device__ __forceinline__ void beside_masked_pass(const Row<T>& row, T* dz, const Range& in, float scale,
                                                   const Factor& f, const Scale& c) {
  constexpr int n = Vec<T>::n;
#pragma unroll 1
  for (int v = in.lo + static_cast<int>(threadIdx.x); v < in.hi; v += NT) {
    if (!row.whole(v)) continue;
    float x[n];
    Vec<T>::unpack(load_vec<T, kStream>(row.z + row.column(v)), x);
#pragma unroll
    for (int e = 0; e < n; ++e) x[e] = x[e] <= c.low ? -kInf : x[e];
    store_whole(dz, row, v, gradient_of<T, kEntropy, kFrom>(Vec<T>::pack(x), scale, f, c));
  }
}

// The gradient of the tiles of `in`, the first of which has been requested into
// r.
template <typename T, int NT, int U, bool kEntropy, int kFrom>
__device__ __forceinline__ void gradient_pass(const Row<T>& row, T* dz, const Range& in, float scale,
                                              const Factor& f, const Scale& c, Raw (&r)[U]) {
  if (beside_masked<kFrom>(f)) {
    beside_masked_pass<T, NT, kEntropy, kFrom>(row, dz, in, scale, f, c);
    return;
  }
  for (int first = in.lo; first < in.hi;) {
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = gradient_of<T, kEntropy, kFrom>(r[u], scale, f, c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = first + u * NT + static_cast<int>(threadIdx.x);
      if (row.whole(v)) store_whole(dz, row, v, r[u]);
    }
    first += NT * U;
    if (first < in.hi) load_tile<T, NT, U, kStream>(row, first, r);
  }
}

// A column outside the whole vectors, in the thread that takes it.
template <typename T>
struct Single {
  int column;  // -1: none
  T z;

  __device__ __forceinline__ void load(const Row<T>& row, const Range& in) {
    column = row.edge();
    if (!holds(row, in, column)) column = -1;
    z = T{};
    if (column >= 0) z = row.z[column];
  }
  __device__ __forceinline__ float logit() const { return column >= 0 ? load_one(&z) : -kInf; }
  template <bool kEntropy, int kFrom>
  __device__ __forceinline__ void gradient(T* dz, float scale, const Factor& f, const Scale& c) const {
    if (column < 0) return;
    const uint32_t word = logit() <= c.low ? Vec<T>::gone : as_word(z);  // the same zeros as in a vector
    dz[column] = from_word<T>(gradient_of<T, kEntropy, kFrom>(Raw{word, 0u, 0u, 0u}, scale, f, c)[0]);
  }
};

// Zeros, or with nan: NaN where the row is not masked.
template <typename T, int NT>
__device__ __forceinline__ void flat_pass(const Row<T>& row, T* dz, const Range& in, bool nan, const Scale& c) {
  constexpr int n = Vec<T>::n;
  const auto flat = [&](float x) { return nan && !(x <= c.low) ? __builtin_nanf("") : 0.0f; };
  const int edge = row.edge();
  if (holds(row, in, edge)) store_one(dz + edge, flat(nan ? load_one(row.z + edge) : 0.0f));
  for (int v = in.lo + static_cast<int>(threadIdx.x); v < in.hi; v += NT) {
    if (!row.whole(v)) continue;
    float x[n] = {};
    if (nan) Vec<T>::unpack(load_vec<T, kStream>(row.z + row.column(v)), x);
#pragma unroll
    for (int e = 0; e < n; ++e) x[e] = flat(x[e]);
    store_whole(dz, row, v, Vec<T>::pack(x));
  }
}

// dz = scale p (-g - h (s - L + H)) with one exponential a logit, the token's
// column after the pass. Bound by HBM: 4096 x 65537 bf16 takes 206 us (5.2 TB/s,
// 94 % of a copy's rate), the vector unit 0.37 busy.
template <typename T, int NT, int U, bool kEntropy>
__global__ __launch_bounds__(NT) void token_logprobs_backward_kernel(LogitsLaunch a, Cut cut) {
  const int64_t at = blockIdx.x / cut.parts;
  T* dz = static_cast<T*>(a.dz) + at * a.lddz;
  const Row<T> row = row_at(static_cast<const T*>(a.z) + at * a.ldz, a.vocab, dz);
  const Range in = range_of<NT, U>(cut, static_cast<int>(blockIdx.x % cut.parts), row.vectors());
  const Scale c = scale_of(a.scale);
  const float lse = a.in_lse[at], ent = kEntropy ? a.in_entropy[at] : 0.0f;
  const int64_t token = a.d_logp ? a.tokens[at] : -1;
  const float g_token = a.d_logp ? a.d_logp[at] : 0.0f;
  const float h = kEntropy ? a.d_entropy[at] : 0.0f;
  const bool mine = threadIdx.x == 0 && holds(row, in, token);
  float x_token = 0.0f;
  Single<T> single;
  single.load(row, in);
  Raw r[U];
  load_tile<T, NT, U, kStream>(row, in.lo, r);
  if (mine) x_token = load_one(row.z + token);
  const float g = token >= 0 ? g_token : 0.0f;
  if ((g == 0.0f && h == 0.0f) || lse == -kInf) {
    flat_pass<T, NT>(row, dz, in, false, c);
    return;
  }
  Factor f;
  f.ref = lse;
  f.b = -h * a.scale;
  f.a = -(g + (h != 0.0f ? h * ent : 0.0f)) * a.scale;
  const float sure = f.a + f.b + lse;
  if (sure - sure != 0.0f || (token >= a.vocab && g != 0.0f)) {
    flat_pass<T, NT>(row, dz, in, true, c);
    return;
  }
  __syncthreads();  // in place: every thread has requested what it reads of others' columns
  gradient_pass<T, NT, U, kEntropy, kFromLse>(row, dz, in, a.scale, f, c, r);
  single.template gradient<kEntropy, kFromLse>(dz, a.scale, f, c);
  __syncthreads();
  if (mine) {  // the token's own column
    const float lp = fma_(x_token, a.scale, -lse), p = exp2_hw(lp * kLog2e);
    const float own = fma_(p, kEntropy ? fma_(lp, f.b, f.a) : f.a, g * a.scale);
    store_one(dz + token, x_token <= c.low ? 0.0f : own);
  }
}

// ---------------------------------------------------------------------------
// Distillation
// ---------------------------------------------------------------------------

// What all threads have to know of a row's alternatives.
struct Taught {
  float rest;     // the teacher's remaining mass
  float masses;   // its other mass
  float over;     // masses - 1 (renormalised: 0)
  Sum members;    // the student's logits, each column once
  int bad;        // an id lies beyond the row
  int doubled;    // an id may be named twice
};

// One row's teacher, in LDS.
struct __attribute__((aligned(16))) Teacher {
  int id[NVFP4_LOGITS_MAX_K];      // -1 where absent or out of range, and from k on
  float q[NVFP4_LOGITS_MAX_K];     // mass
  float ln_q[NVFP4_LOGITS_MAX_K];
  uint8_t slot[512];               // of are_different
  Taught m;
};

// The alternatives are the first wave's business, two a lane (lane and lane +
// 64): it needs no barrier for them, and the other waves go on with the row.
constexpr int kOwn = NVFP4_LOGITS_MAX_K / 64;

struct Alternatives {
  int id[kOwn];    // as given; -1 in the other waves
  float a[kOwn];   // log probability
  float x[kOwn];   // the student's logit; -inf where there is none, or it is not wanted
};

// wanted(id): whether the caller uses the logit of id. A part of a row reads no
// others': the gradient of 64 rows of 32768 float32 logits (8.4 MB) with 128
// alternatives reads 9.1 MB so, and 16.0 with all of them; and in place the other
// parts overwrite theirs meanwhile.
template <typename T, typename F>
__device__ __forceinline__ Alternatives load_alternatives(const LogitsLaunch& a, const T* z, int64_t at, F wanted) {
  Alternatives m;
#pragma unroll
  for (int h = 0; h < kOwn; ++h) {
    const int j = threadIdx.x + 64 * h;
    m.id[h] = -1;
    m.a[h] = m.x[h] = -kInf;
    if (threadIdx.x < 64 && j < a.k) {
      m.id[h] = a.t_ids[at * a.k + j];
      const float lp = a.t_logp[at * a.k + j];
      if (m.id[h] >= 0) m.a[h] = lp;
    }
  }
#pragma unroll
  for (int h = 0; h < kOwn; ++h)
    if (m.id[h] >= 0 && m.id[h] < a.vocab && wanted(m.id[h])) m.x[h] = load_one(z + m.id[h]);
  return m;
}

// Whether an earlier alternative than j names `id` (j = k: any).
__device__ __forceinline__ bool named_before(const Teacher& t, int id, int j) {
  bool found = false;
  for (int i = 0; i < j; i += 4) {
    const int4 four = *reinterpret_cast<const int4*>(&t.id[i]);
    found |= four.x == id | (i + 1 < j & four.y == id) | (i + 2 < j & four.z == id) | (i + 3 < j & four.w == id);
  }
  return found;
}

// Whether the column is an alternative, k of which have been named.
__device__ __forceinline__ bool is_named(const Teacher& t, int64_t column, int k) {
  return named_before(t, static_cast<int>(column), k);
}

// Names the alternatives, as teach does (for the first wave).
__device__ __forceinline__ void name(const Alternatives& own, Teacher& t) {
#pragma unroll
  for (int h = 0; h < kOwn; ++h) t.id[threadIdx.x + 64 * h] = own.id[h];
}

// What the first wave has written to LDS so far is there for its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Whether the wave's ids (those >= 0 of t.id) are all different (false: perhaps
// not). Each round the ids go to slots by a hash; who finds its own index there
// is through, who finds its own id under another index ends the search, the
// others go on. 128 different ids in 512 slots: about 15 are left after a round,
// seldom any after two.
__device__ __forceinline__ bool are_different(Teacher& t) {
  const int lane = threadIdx.x;
  int id[kOwn];
#pragma unroll
  for (int h = 0; h < kOwn; ++h) id[h] = t.id[lane + 64 * h];
  uint32_t factor = 2654435761u;
#pragma unroll 1
  for (int round = 0; round < 4; ++round, factor = factor * 1664525u + 1013904222u | 1u) {
    uint32_t at[kOwn];
#pragma unroll
    for (int h = 0; h < kOwn; ++h) {
      at[h] = (static_cast<uint32_t>(id[h]) * factor) >> 23;
      if (id[h] >= 0) t.slot[at[h]] = static_cast<uint8_t>(lane + 64 * h);
    }
    wave_sync();
    bool any = false, same = false;
#pragma unroll
    for (int h = 0; h < kOwn; ++h) {
      const int there = t.slot[at[h]];
      if (there == lane + 64 * h) id[h] = -1;  // through
      any |= id[h] >= 0;
      same |= id[h] >= 0 && t.id[there & (NVFP4_LOGITS_MAX_K - 1)] == id[h];
    }
    if (__ballot(same) != 0) return false;
    if (__ballot(any) == 0) return true;
    wave_sync();
  }
  return false;
}

// Fills t from the alternatives; kSums: members and ln_q too. For the first
// wave alone; a barrier later the others may read it. Nothing here needs the
// row's sum, so it runs while the row's first logits are on their way. What the
// masses leave of 1 is formed in 64 bits: it may be far below float32's u, and
// a loss near 0 consists of such differences.
template <bool kSums>
__device__ __forceinline__ void teach(const LogitsLaunch& a, const Alternatives& own, Teacher& t, const Scale& c) {
  float rest = a.tail ? 1.0f : 0.0f, masses = 0.0f, over = 0.0f;
  Sum members = {kNoRef, 0.0f, 0.0f};
  bool bad = false, doubled = false;
  const int lane = threadIdx.x;
  if (a.k > 0) {
    float q[kOwn], ln_q[kOwn], top = -kInf, sum = 0.0f;
    bool beyond = false;
#pragma unroll
    for (int h = 0; h < kOwn; ++h) {
      beyond |= own.id[h] >= a.vocab;
      top = fmaxf(top, own.a[h]);
    }
    bad = __ballot(beyond) != 0;
#pragma unroll
    for (int h = 0; h < kOwn; ++h) t.id[lane + 64 * h] = own.id[h] >= a.vocab ? -1 : own.id[h];
    wave_sync();
    doubled = !are_different(t);
    top = wave_max(top);
    if (a.tail || top == -kInf) top = 0.0f;
    if (a.tail) {
      double all = 0.0;
#pragma unroll
      for (int h = 0; h < kOwn; ++h) {
        ln_q[h] = own.a[h];
        const double e = exp(static_cast<double>(own.a[h]));
        q[h] = static_cast<float>(e);
        all += e;
      }
      all = wave_sum(all);
      masses = static_cast<float>(all);
      over = static_cast<float>(all - 1.0);
      rest = all > 1.0 - kLeastTail ? 0.0f : static_cast<float>(1.0 - all);
    } else {
#pragma unroll
      for (int h = 0; h < kOwn; ++h) {
        ln_q[h] = own.a[h] - top;
        q[h] = expf(ln_q[h]);
        sum += q[h];
      }
      masses = wave_sum(sum);
      if (masses > 0.0f) {
        const float ln_sum = logf(masses);
#pragma unroll
        for (int h = 0; h < kOwn; ++h) {
          q[h] /= masses;
          ln_q[h] -= ln_sum;
        }
        masses = 1.0f;
      }
    }
#pragma unroll
    for (int h = 0; h < kOwn; ++h) t.q[lane + 64 * h] = q[h];
    if (kSums) {
      Running run = running(c);
#pragma unroll
      for (int h = 0; h < kOwn; ++h) {
        const int id = t.id[lane + 64 * h];
        if (id >= 0 && !(doubled && named_before(t, id, lane + 64 * h))) add_one<false>(run, own.x[h], c);
      }
      members = wave_join(finished(run));
#pragma unroll
      for (int h = 0; h < kOwn; ++h) t.ln_q[lane + 64 * h] = ln_q[h];
    }
  } else {
#pragma unroll
    for (int h = 0; h < kOwn; ++h) t.id[lane + 64 * h] = -1;
  }
  if (lane == 0) {
    t.m.rest = rest;
    t.m.masses = masses;
    t.m.bad = bad;
    t.m.doubled = doubled;
    t.m.over = over;
    if (kSums) t.m.members = members;
  }
}

// The whole mass of `id` (0: not named).
__device__ __forceinline__ float mass_of(const Teacher& t, int id, int k) {
  float q = 0.0f;
  for (int i = 0; i < k; i += 4) {
    const int4 four = *reinterpret_cast<const int4*>(&t.id[i]);
    const float4 mass = *reinterpret_cast<const float4*>(&t.q[i]);
    q += (four.x == id ? mass.x : 0.0f) + (four.y == id ? mass.y : 0.0f) + (four.z == id ? mass.z : 0.0f) +
         (four.w == id ? mass.w : 0.0f);
  }
  return q;
}

// The alternatives of a tile are marked in LDS, a bit per logit and 8 bits per
// vector, U of them per thread. A tile's marks are in one of two buffers: the
// owner clears what it finds, so the other buffer is clean again when its turn
// comes, two barriers later.
template <int NT, int U, int kBuffers = 2>
struct Marks {
  static constexpr int words = (U + 3) / 4;
  uint32_t word[kBuffers][words * NT];
  uint32_t singles;  // of the columns outside the whole vectors, by the thread that takes them

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < kBuffers; ++b)
#pragma unroll
      for (int h = 0; h < words; ++h) word[b][words * threadIdx.x + h] = 0;
    if (threadIdx.x == 0) singles = 0;
    __syncthreads();
  }
  // Whether the thread's single column is an alternative.
  __device__ __forceinline__ bool single() const { return singles >> threadIdx.x & 1u; }
  // Marks the ids among the single columns.
  template <typename T>
  __device__ __forceinline__ void put_singles(const Row<T>& row, const Alternatives& own) {
#pragma unroll
    for (int h = 0; h < kOwn; ++h) {
      const int taker = row.taker(own.id[h]);
      if (taker >= 0) atomicOr(&singles, 1u << taker);
    }
  }
  // Marks the ids in the tile at `first`; gone: the thread's marks.
  template <typename T>
  __device__ __forceinline__ void take(const Row<T>& row, const Alternatives& own, int first, int buffer,
                                       uint32_t (&gone)[words]) {
    constexpr int n = Vec<T>::n;
#pragma unroll
    for (int h = 0; h < kOwn; ++h) {
      if (own.id[h] < 0 || own.id[h] >= row.vocab) continue;
      const int64_t p = static_cast<int64_t>(own.id[h]) + row.skip;
      const int at = static_cast<int>(p / n) - first;
      if (at >= 0 && at < NT * U) {
        const int u = at / NT, owner = at % NT;
        atomicOr(&word[buffer][words * owner + (u >> 2)], 1u << (8 * (u & 3) + static_cast<int>(p % n)));
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < words; ++h) {
      uint32_t& mine = word[buffer][words * threadIdx.x + h];
      gone[h] = mine;
      if (gone[h]) mine = 0;
    }
  }
};

// Adds a vector without its marked logits.
template <typename T>
__device__ __forceinline__ void add_unmarked(Running& run, const Raw& r, uint32_t marks, const Scale& c) {
  constexpr int n = Vec<T>::n;
  float x[n];
  Vec<T>::unpack(r, x);
  if (marks) {
#pragma unroll
    for (int e = 0; e < n; ++e) x[e] = marks >> e & 1u ? -kInf : x[e];
  }
  add_logits<false>(run, x, max_of(x), c);
}

// Adds the tiles of `in` without the alternatives, the first tile of which has
// been requested into r.
template <typename T, int NT, int U, int kHow>
__device__ __forceinline__ void add_tail(Running& run, const LogitsLaunch& a, const Row<T>& row,
                                         const Alternatives& own, const Range& in, const Scale& c,
                                         Marks<NT, U>& marks, Raw (&r)[U]) {
  int buffer = 0;
  for (int first = in.lo; first < in.hi; buffer ^= 1) {
    uint32_t gone[Marks<NT, U>::words] = {};
    if (a.k > 0) marks.take(row, own, first, buffer, gone);
    const int used = used_of<NT, U>(first, in.hi);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < used) add_unmarked<T>(run, r[u], gone[u >> 2] >> (8 * (u & 3)) & 0xFFu, c);
    first += NT * U;
    if (first < in.hi) load_tile<T, NT, U, kHow>(row, first, r);
  }
}

// A row's sums.
struct RowSums {
  Sum tail, whole;
};

// q (d - 1) + p for masses q > 0 and p = q e^-d: not negative, and near d = 0,
// where its parts cancel, from the series q (d^2/2! - d^3/3! + ...). At |d| = 1
// the last term left out is 1e-8 of it, and the other form has 7 u.
__device__ __forceinline__ float excess(float q, float d, float p) {
  if (fabsf(d) > 1.0f) return fma_(q, d - 1.0f, p);
  float g = 1.0f / 39916800.0f;  // 11!
  g = fma_(g, -d, 1.0f / 3628800.0f);
  g = fma_(g, -d, 1.0f / 362880.0f);
  g = fma_(g, -d, 1.0f / 40320.0f);
  g = fma_(g, -d, 1.0f / 5040.0f);
  g = fma_(g, -d, 1.0f / 720.0f);
  g = fma_(g, -d, 1.0f / 120.0f);
  g = fma_(g, -d, 1.0f / 24.0f);
  g = fma_(g, -d, 1.0f / 6.0f);
  g = fma_(g, -d, 0.5f);
  return q * (d * d * g);
}

// The row's divergence, in lane 0 of the first wave, which alone calls this. With
// d = ln (q / p) the terms q d cancel where the student is near its teacher;
// excess(q, d, p) = q d - q + p do not. Their sum lacks Q - P, the teacher's mass
// on the terms less the student's. All of the student's masses together are 1,
// so of P only what counts not once is added up: columns named without mass, or
// twice, and the tail where it is no term.
__device__ __forceinline__ float divergence(const Alternatives& own, const Sum& whole, const Sum& tail,
                                            const Teacher& t, const Scale& c) {
  const Taught& m = t.m;
  const int lane = threadIdx.x;
  const Log2 l = split_log2(whole.s);
  float part = 0.0f;
#pragma unroll
  for (int h = 0; h < kOwn; ++h) {
    const int j = lane + 64 * h, id = t.id[j];
    const float q = t.q[j], y = fma_(own.x[h], c.c, -whole.r);
    const bool live = own.x[h] > c.low;  // not so for an absent one
    const float p = live ? exp2_hw(y) / whole.s : 0.0f;
    const bool term = q != 0.0f, once = live && !(m.doubled && named_before(t, id, j));
    if (term) part += excess(q, live ? t.ln_q[j] - ((y - l.whole) - l.left) * kLn2Hi : kInf, p);
    if (term != once) part += once ? p : -p;
  }
  float loss = wave_sum(part);
  const float p_rest = tail.s == 0.0f ? 0.0f : exp2_hw(shift_of(tail.r, whole.r)) * (tail.s / whole.s);
  if (m.rest > 0.0f) {
    const Log2 r = split_log2(tail.s);
    const float lp = ((tail.r - whole.r) + (r.whole - l.whole)) + (r.left - l.left);
    loss += excess(m.rest, tail.s == 0.0f ? kInf : logf(m.rest) - lp * kLn2Hi, p_rest);
  } else if (m.masses == 0.0f) {
    loss = 0.0f;  // a teacher without mass
  } else {
    loss += m.over + p_rest;
  }
  return loss;
}

// Joins the alternatives to the tail and writes the row's outputs.
__device__ __forceinline__ RowSums finish_distill(const LogitsLaunch& a, int64_t at, int64_t token, float x_token,
                                                  const Sum& tail, const Alternatives& own, const Teacher& t,
                                                  const Scale& c) {
  const RowSums s = {tail, a.k > 0 ? join(tail, t.m.members) : tail};
  float loss = 0.0f;
  if (a.k > 0 && threadIdx.x < 64) loss = divergence(own, s.whole, tail, t, c);
  if (threadIdx.x == 0) {
    const float l2 = log2_hw(s.whole.s), tail_l2 = log2_hw(tail.s);
    bool bad = s.whole.s != s.whole.s || t.m.bad;
    if (bad) loss = __builtin_nanf("");
    a.loss[at] = loss;
    a.lse[at] = s.whole.s == 0.0f ? -kInf : to_nats(s.whole.r, l2);
    a.lse_tail[at] = tail.s == 0.0f ? -kInf : to_nats(tail.r, tail_l2);
    if (a.logp) a.logp[at] = token_logp(a.vocab, token, x_token, c, s.whole, l2, &bad);
    if (bad && a.dev_status) *a.dev_status = 1;
  }
  return s;
}

// The sum of the columns that are no alternative, from a bit per logit in LDS;
// the alternatives' part comes from the first wave. Bound by HBM: 2048 x 131072
// bf16 with 64 alternatives takes 84 us (6.4 TB/s, 96 % of a read's rate at that
// size), the vector unit 0.61 busy.
template <typename T, int NT, int U>
__global__ __launch_bounds__(NT) void distill_kernel(LogitsLaunch a, Cut cut) {
  __shared__ Teacher teacher;
  __shared__ Shared<NT> lds;
  __shared__ Marks<NT, U> marks;
  const int64_t at = blockIdx.x / cut.parts;
  const T* z = static_cast<const T*>(a.z) + at * a.ldz;
  const Row<T> row = row_at(z, a.vocab, z);
  const Range in = range_of<NT, U>(cut, static_cast<int>(blockIdx.x % cut.parts), row.vectors());
  const Scale c = scale_of(a.scale);
  const Alternatives own = load_alternatives(a, z, at, [&](int) { return cut.parts == 1; });
  float x_token;
  const int64_t token = load_token(a, z, at, &x_token);
  Single<T> single;
  single.load(row, in);
  Raw r[U];
  load_tile<T, NT, U, kStream>(row, in.lo, r);
  if (threadIdx.x < 64) {
    if (cut.parts == 1) teach<true>(a, own, teacher, c);
    else name(own, teacher);
  }
  marks.clear();
  marks.put_singles(row, own);
  Running run = running(c);
  add_tail<T, NT, U, kStream>(run, a, row, own, in, c, marks, r);
  without_masked<T, NT, false>(run, row, in, c, [&](int64_t column) { return is_named(teacher, column, a.k); });
  if (a.k > 0) __syncthreads();  // a part without tiles has had none since put_singles
  if (single.column >= 0 && !marks.single()) add_one<false>(run, single.logit(), c);
  const Sum t = block_join(finished(run), lds);
  if (cut.parts > 1) {
    if (threadIdx.x == 0) part_sums(a)[blockIdx.x] = Part{t.r, t.s, 0.0f, 0.0f};
    return;
  }
  finish_distill(a, at, token, x_token, t, own, teacher, c);
}

// Finishes rows that were cut into parts: 4.6 us, most of it a launch's latency.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void distill_join_kernel(LogitsLaunch a, Cut cut) {
  __shared__ Teacher teacher;
  __shared__ Shared<NT> lds;
  const int64_t at = blockIdx.x;
  const T* z = static_cast<const T*>(a.z) + at * a.ldz;
  const Scale c = scale_of(a.scale);
  const Alternatives own = load_alternatives(a, z, at, [](int) { return true; });
  float x_token;
  const int64_t token = load_token(a, z, at, &x_token);
  if (threadIdx.x < 64) teach<true>(a, own, teacher, c);
  const Sum t = join_parts(a, at, cut, lds);  // its barriers: teacher.m is there
  finish_distill(a, at, token, x_token, t, own, teacher, c);
}

// Upstream gradients of a row.
struct Upstream {
  float gk, gl;
  int64_t label;

  // gk v; 0 where the teacher has no weight, whatever it holds
  __device__ __forceinline__ float of_teacher(float v) const { return gk != 0.0f ? gk * v : 0.0f; }
};

__device__ __forceinline__ Upstream upstream(const LogitsLaunch& a, int64_t at) {
  Upstream g;
  g.label = a.d_logp ? a.tokens[at] : -1;
  g.gl = g.label >= 0 ? a.d_logp[at] : 0.0f;
  g.gk = a.d_loss ? a.d_loss[at] : 0.0f;
  return g;
}

// Whether the row's gradient is NaN: by an index beyond the row, or by f.
__device__ __forceinline__ bool is_nan_row(const LogitsLaunch& a, const Taught& m, const Upstream& g,
                                           const Factor& f) {
  const float sure = f.a + f.ref;
  return (m.bad && g.gk != 0.0f) || (g.label >= a.vocab && g.gl != 0.0f) || sure - sure != 0.0f;
}

// Columns whose gradient a lane of the first wave writes after the pass (-1:
// none): its alternatives, and lane 0 the label.
struct Special {
  int column[kOwn], label;
  float value[kOwn], of_label;

  template <typename T>
  __device__ __forceinline__ void write(T* dz) const {
#pragma unroll
    for (int h = 0; h < kOwn; ++h)
      if (column[h] >= 0) store_one(dz + column[h], value[h]);
    if (label >= 0) store_one(dz + label, of_label);
  }
};

// prob(x): an alternative's probability; x_label: the label's logit in lane 0,
// rest_of(x_label): its gradient without the label's term. Masses of an id named
// twice add up.
template <typename T, typename P, typename Q>
__device__ __forceinline__ Special special_columns(const LogitsLaunch& a, const Row<T>& row, const Range& in,
                                                   const Alternatives& own, const Teacher& t, const Upstream& g,
                                                   float x_label, const Scale& c, P prob, Q rest_of) {
  Special s;
  const float all = t.m.masses + t.m.rest;
  const bool doubled = t.m.doubled;
  bool among = false;
#pragma unroll
  for (int h = 0; h < kOwn; ++h) {
    const int id = own.id[h];
    const bool here = holds(row, in, id);  // not in the other waves: -1
    among |= id >= 0 && id == g.label;
    float v = 0.0f;
    if (here && !(own.x[h] <= c.low)) {
      const float p = prob(own.x[h]);
      const float q = doubled ? mass_of(t, id, a.k) : t.q[(threadIdx.x & 63) + 64 * h];
      v = (g.of_teacher(all * p - q) + g.gl * ((id == g.label ? 1.0f : 0.0f) - p)) * a.scale;
    }
    s.column[h] = here ? id : -1;
    s.value[h] = v;
  }
  const bool alone = __ballot(among) == 0 && threadIdx.x == 0 && holds(row, in, g.label);
  s.label = alone ? static_cast<int>(g.label) : -1;
  s.of_label = x_label <= c.low ? 0.0f : rest_of(x_label) + g.gl * a.scale;
  return s;
}

// One exponential a logit with the row's factor, the label's and the
// alternatives' columns after the pass. Bound by HBM: 4096 x 100003 bf16 with 32
// alternatives takes 320 us (5.1 TB/s, 93 % of a copy's rate).
template <typename T, int NT, int U>
__global__ __launch_bounds__(NT) void distill_backward_kernel(LogitsLaunch a, Cut cut) {
  __shared__ Teacher teacher;
  __shared__ Shared<NT> lds;
  const int64_t at = blockIdx.x / cut.parts;
  const T* z = static_cast<const T*>(a.z) + at * a.ldz;
  T* dz = static_cast<T*>(a.dz) + at * a.lddz;
  const Row<T> row = row_at(z, a.vocab, dz);
  const Range in = range_of<NT, U>(cut, static_cast<int>(blockIdx.x % cut.parts), row.vectors());
  const Scale c = scale_of(a.scale);
  const Upstream g = upstream(a, at);
  const float lse = a.in_lse[at], lse_tail = a.in_lse_tail ? a.in_lse_tail[at] : lse;
  if ((g.gl == 0.0f && g.gk == 0.0f) || lse == -kInf) {
    flat_pass<T, NT>(row, dz, in, false, c);
    return;
  }
  const Alternatives own = load_alternatives(a, z, at, [&](int id) { return holds(row, in, id); });
  float x_label = 0.0f;
  if (threadIdx.x == 0 && holds(row, in, g.label)) x_label = load_one(z + g.label);
  Single<T> single;
  single.load(row, in);
  Raw r[U];
  load_tile<T, NT, U, kStream>(row, in.lo, r);
  if (threadIdx.x < 64) teach<false>(a, own, teacher, c);
  __syncthreads();
  const Taught m = teacher.m;
  // Outside the alternatives d = e^(s - L) (gk all - gl) - gk rest e^(s - L_r)
  // = e^(s - L_r) ((gk all - gl) e^(L_r - L) - gk rest): one exponential, and
  // no factor above 1, however little of the student's mass lies there.
  const bool from_tail = m.rest != 0.0f && g.gk != 0.0f && lse_tail != -kInf;
  const float ref = from_tail ? lse_tail : lse, both = g.of_teacher(m.masses + m.rest) - g.gl;
  const float factor = (from_tail ? both * expf(lse_tail - lse) - g.gk * m.rest : both) * a.scale;
  const Factor f = {factor, 0.0f, ref};
  if (is_nan_row(a, m, g, f)) {
    flat_pass<T, NT>(row, dz, in, true, c);
    return;
  }
  gradient_pass<T, NT, U, false, kFromLse>(row, dz, in, a.scale, f, c, r);
  single.template gradient<false, kFromLse>(dz, a.scale, f, c);
  const float scale = a.scale;
  const auto p_of = [scale](float x, float ref) { return exp2_hw(fma_(x, scale, -ref) * kLog2e); };
  const Special after = special_columns(
      a, row, in, own, teacher, g, x_label, c, [=](float x) { return p_of(x, lse); },
      [=](float x) { return p_of(x, ref) * factor; });
  __syncthreads();
  after.write(dz);
}

// Loss and gradient of whole rows. A workgroup holds the row's first U vectors
// a thread in registers between the sums and the gradient, so they are read
// once: 16 waves of 16 vectors a lane hold 256 KB on a CU. What a longer row
// has beyond them (kMore) is read twice, 4 vectors a thread at a time. 2048 x
// 65536 bf16 takes 95 us (5.6 TB/s, a copy's rate), 8192 x 131072 with 64
// alternatives 896 (4.8 TB/s, 89 %): 1024 threads have a CU to themselves there,
// so loads, reduction and stores overlap only from one row to the next. In two
// passes it took 1275; 512 threads that hold half a row 915 to 970.
template <typename T, int NT, int U, bool kMore>
__global__ __launch_bounds__(NT) void distill_step_kernel(LogitsLaunch a) {
  constexpr int n = Vec<T>::n, more = 4;
  __shared__ Teacher teacher;
  __shared__ Shared<NT> lds;
  __shared__ Marks<NT, U, 1> marks;
  __shared__ Marks<kMore ? NT : 64, more> more_marks;
  const int64_t at = blockIdx.x;
  const T* z = static_cast<const T*>(a.z) + at * a.ldz;
  T* dz = static_cast<T*>(a.dz) + at * a.lddz;
  const Row<T> row = row_at(z, a.vocab, z);
  const Range in = {0, row.vectors()}, rest = {NT * U, in.hi};
  // held vectors count from the line, or where that leaves no room for the last
  // whole vectors from the first whole one
  const int first = kMore || in.hi <= NT * U ? 0 : (row.skip + n - 1) / n;
  const Scale c = scale_of(a.scale);
  const Alternatives own = load_alternatives(a, z, at, [](int) { return true; });
  float x_token;
  const int64_t token = load_token(a, z, at, &x_token);
  const Upstream g = upstream(a, at);
  float x_label = 0.0f;
  if (threadIdx.x == 0 && g.label >= 0 && g.label < a.vocab) x_label = load_one(z + g.label);
  Single<T> single;
  single.load(row, in);
  Raw r[U];
  load_tile<T, NT, U, kStream>(row, first, r);
  if (threadIdx.x < 64) teach<true>(a, own, teacher, c);
  marks.clear();
  uint32_t gone[Marks<NT, U, 1>::words] = {};
  if (a.k > 0) {
    marks.put_singles(row, own);
    marks.take(row, own, first, 0, gone);
  }
  Running run = running(c);
  const int used = used_of<NT, U>(first, in.hi);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < used) add_unmarked<T>(run, r[u], gone[u >> 2] >> (8 * (u & 3)) & 0xFFu, c);
  if constexpr (kMore) {
    more_marks.clear();
    Raw q[more];
    load_tile<T, NT, more, kKeep>(row, rest.lo, q);
    add_tail<T, NT, more, kKeep>(run, a, row, own, rest, c, more_marks, q);
  }
  without_masked<T, NT, false>(run, row, Range{first, in.hi}, c,
                               [&](int64_t column) { return is_named(teacher, column, a.k); });
  if (single.column >= 0 && !marks.single()) add_one<false>(run, single.logit(), c);
  const Sum t = block_join(finished(run), lds);
  const Taught m = teacher.m;
  const RowSums s = finish_distill(a, at, token, x_token, t, own, teacher, c);
  if ((g.gl == 0.0f && g.gk == 0.0f) || s.whole.s == 0.0f) {
    flat_pass<T, NT>(row, dz, in, false, c);
    return;
  }
  // as in the backward kernel, with the sums themselves; without a tail against
  // the whole, above which no logit lies far (a masked one does above kNoRef)
  const float ref = t.s != 0.0f ? t.r : s.whole.r;
  const float share = exp2_hw(shift_of(ref, s.whole.r)) / s.whole.s;
  Factor f = {(g.of_teacher(m.masses + m.rest) - g.gl) * share, 0.0f, ref};
  if (m.rest != 0.0f && g.gk != 0.0f && t.s != 0.0f) f.a -= g.gk * m.rest / t.s;
  f.a *= a.scale;
  if (is_nan_row(a, m, g, f)) {
    flat_pass<T, NT>(row, dz, in, true, c);
    return;
  }
  // by the first wave, while the others store
  const Special after = special_columns(
      a, row, in, own, teacher, g, x_label, c,
      [&](float x) { return exp2_hw(fma_(x, c.c, -s.whole.r)) / s.whole.s; },
      [&](float x) { return exp2_hw(fma_(x, c.c, -f.ref)) * f.a; });
  if (beside_masked<kFromRef>(f)) {
    beside_masked_pass<T, NT, false, kFromRef>(row, dz, Range{first, in.hi}, a.scale, f, c);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = first + u * NT + static_cast<int>(threadIdx.x);
      if (row.whole(v)) store_whole(dz, row, v, gradient_of<T, false, kFromRef>(r[u], a.scale, f, c));
    }
    if constexpr (kMore) {
      Raw q[more];
      load_tile<T, NT, more, kStream>(row, rest.lo, q);
      gradient_pass<T, NT, more, false, kFromRef>(row, dz, rest, a.scale, f, c, q);
    }
  }
  single.template gradient<false, kFromRef>(dz, a.scale, f, c);
  __syncthreads();
  after.write(dz);
}

// Rows of one launch (the grid's work items fit 32 bits).
constexpr int64_t kRowsPerLaunch = 1 << 21;

LogitsLaunch rows_from(const LogitsLaunch& a, int64_t r) {
  LogitsLaunch b = a;
  const int64_t size = a.z_bf16 ? 2 : 4;
  auto at = [&](auto* p, int64_t n) { return p ? p + n : p; };
  b.z = static_cast<const char*>(a.z) + r * a.ldz * size;
  b.dz = a.dz ? static_cast<char*>(a.dz) + r * a.lddz * size : nullptr;
  b.rows = a.rows - r < kRowsPerLaunch ? a.rows - r : kRowsPerLaunch;
  b.tokens = at(a.tokens, r);
  b.t_ids = at(a.t_ids, r * a.k);
  b.t_logp = at(a.t_logp, r * a.k);
  b.logp = at(a.logp, r);
  b.entropy = at(a.entropy, r);
  b.lse = at(a.lse, r);
  b.lse_tail = at(a.lse_tail, r);
  b.loss = at(a.loss, r);
  b.top_ids = at(a.top_ids, r * a.k);
  b.top_logp = at(a.top_logp, r * a.k);
  b.in_lse = at(a.in_lse, r);
  b.in_entropy = at(a.in_entropy, r);
  b.in_lse_tail = at(a.in_lse_tail, r);
  b.d_logp = at(a.d_logp, r);
  b.d_entropy = at(a.d_entropy, r);
  b.d_loss = at(a.d_loss, r);
  return b;
}

template <typename F>
int by_rows(const LogitsLaunch& a, F launch) {
  for (int64_t r = 0; r < a.rows; r += kRowsPerLaunch) {
    launch(rows_from(a, r));
    if (hipGetLastError() != hipSuccess) return -1;
  }
  return 0;
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

// Workgroup shapes: threads, and vectors a thread has in flight.
struct Long {  // many rows
  static constexpr int threads = 256, unroll = 8;
};
struct Short {  // short rows, and parts of few rows
  static constexpr int threads = 256, unroll = 2;
};
struct Wide {  // whole rows of a few
  static constexpr int threads = 1024, unroll = 8;
};
enum Shape { kLong, kShort, kWide };

struct Plan {
  Shape shape;
  Cut cut;
};

int64_t tile_of(Shape s) {
  return s == kLong ? Long::threads * Long::unroll : s == kWide ? Wide::threads * Wide::unroll : Short::threads * Short::unroll;
}

// `parts` workgroups a row at most.
Plan cut_rows(Shape shape, int64_t vectors, int64_t parts) {
  const int64_t tiles = (vectors + tile_of(shape) - 1) / tile_of(shape);
  if (parts > tiles) parts = tiles;
  if (parts < 1) parts = 1;
  const int64_t each = (tiles + parts - 1) / parts;
  return Plan{shape, Cut{static_cast<int>((tiles + each - 1) / each), static_cast<int>(each)}};
}

// Vectors of a row: rows that start on a line, or at the worst place.
int64_t vectors_of(bool bf16, int64_t vocab, bool lines) {
  const int64_t n = bf16 ? 8 : 4, skip = lines ? 0 : bf16 ? 63 : 31;
  return (vocab + skip + n - 1) / n;
}

bool on_lines(const void* p, int64_t ld, bool bf16) {
  return reinterpret_cast<uintptr_t>(p) % 128 == 0 && ld * (bf16 ? 2 : 4) % 128 == 0;
}

constexpr int64_t kWantedGroups = 1024, kCus = 256;

// Few rows of up to 512 KB: a wide workgroup each, and no second launch. 131072
// bf16 logits without alternatives then take 9.6 us a call instead of 13.8 (for
// 1 row; 15.8 instead of 18.5 for 256), with 20 alternatives 15.2 instead of
// 16.8 (22.2 instead of 26.5); 50001 logits 12.2 instead of 15.8. From 300 rows
// on their workgroups take turns on the CUs, and parts are as quick.
// Else rows are cut into parts until there are as many workgroups as the GPU
// can have at hand; parts of short tiles where long ones would be too few.
Plan plan_forward(int64_t rows, int64_t vectors) {
  if (vectors <= 2 * tile_of(kShort)) return cut_rows(kShort, vectors, 1);
  if (rows <= kCus && vectors <= 32768) return cut_rows(kWide, vectors, 1);
  const int64_t groups = rows * ((vectors + tile_of(kLong) - 1) / tile_of(kLong));
  return cut_rows(groups >= kWantedGroups ? kLong : kShort, vectors, (kWantedGroups + rows - 1) / rows);
}
Plan plan_forward(const LogitsLaunch& a) {
  return plan_forward(a.rows, vectors_of(a.z_bf16, a.vocab, on_lines(a.z, a.ldz, a.z_bf16)));
}

Plan plan_backward(const LogitsLaunch& a) {
  const int64_t vectors = vectors_of(a.z_bf16, a.vocab, on_lines(a.dz, a.lddz, a.z_bf16));
  const int64_t groups = a.rows * ((vectors + tile_of(kLong) - 1) / tile_of(kLong));
  const Shape shape = groups >= kWantedGroups && vectors > 2 * tile_of(kShort) ? kLong : kShort;
  return cut_rows(shape, vectors, (kWantedGroups + a.rows - 1) / a.rows);
}

// Calls f(T(), shape) for the type and the plan.
template <typename F>
void by_shape(bool bf16, Shape s, F f) {
  const auto with = [&](auto type) {
    if (s == kLong) f(type, Long());
    else if (s == kWide) f(type, Wide());
    else f(type, Short());
  };
  if (bf16) with(uint16_t());
  else with(float());
}

unsigned grid_of(const LogitsLaunch& a, const Plan& p) { return static_cast<unsigned>(a.rows * p.cut.parts); }

}  // namespace

int64_t logits_workspace_bytes(bool z_bf16, int64_t rows, int64_t vocab, int k) {
  if (rows == 0) return 0;
  // the rows' alignment is not known here
  const int parts[2] = {plan_forward(rows, vectors_of(z_bf16, vocab, true)).cut.parts,
                        plan_forward(rows, vectors_of(z_bf16, vocab, false)).cut.parts};
  const int64_t most = parts[0] > parts[1] ? parts[0] : parts[1];
  return most == 1 ? 0 : rows * most * static_cast<int64_t>(sizeof(Part) + sizeof(uint64_t) * k);
}

int launch_token_logprobs(const LogitsLaunch& a, hipStream_t stream) {
  const Plan p = plan_forward(a);
  return by_rows(a, [&](const LogitsLaunch& b) {
    by_shape(b.z_bf16, p.shape, [&](auto type, auto shape) {
      using T = decltype(type);
      constexpr int NT = decltype(shape)::threads, U = decltype(shape)::unroll;
      const dim3 grid(grid_of(b, p)), block(NT);
      if (b.k > 0)
        b.entropy ? token_logprobs_kernel<T, NT, U, true, true><<<grid, block, 0, stream>>>(b, p.cut)
                  : token_logprobs_kernel<T, NT, U, true, false><<<grid, block, 0, stream>>>(b, p.cut);
      else
        b.entropy ? token_logprobs_kernel<T, NT, U, false, true><<<grid, block, 0, stream>>>(b, p.cut)
                  : token_logprobs_kernel<T, NT, U, false, false><<<grid, block, 0, stream>>>(b, p.cut);
      if (p.cut.parts > 1)
        token_logprobs_join_kernel<T, 256><<<static_cast<unsigned>(b.rows), 256, 0, stream>>>(b, p.cut);
    });
  });
}

int launch_token_logprobs_backward(const LogitsLaunch& a, hipStream_t stream) {
  const Plan p = plan_backward(a);
  return by_rows(a, [&](const LogitsLaunch& b) {
    by_shape(b.z_bf16, p.shape, [&](auto type, auto shape) {
      using T = decltype(type);
      constexpr int NT = decltype(shape)::threads, U = decltype(shape)::unroll;
      const dim3 grid(grid_of(b, p)), block(NT);
      b.d_entropy ? token_logprobs_backward_kernel<T, NT, U, true><<<grid, block, 0, stream>>>(b, p.cut)
                  : token_logprobs_backward_kernel<T, NT, U, false><<<grid, block, 0, stream>>>(b, p.cut);
    });
  });
}

int launch_distill(const LogitsLaunch& a, hipStream_t stream) {
  const Plan p = plan_forward(a);
  return by_rows(a, [&](const LogitsLaunch& b) {
    by_shape(b.z_bf16, p.shape, [&](auto type, auto shape) {
      using T = decltype(type);
      constexpr int NT = decltype(shape)::threads, U = decltype(shape)::unroll;
      distill_kernel<T, NT, U><<<grid_of(b, p), NT, 0, stream>>>(b, p.cut);
      if (p.cut.parts > 1)
        distill_join_kernel<T, 256><<<static_cast<unsigned>(b.rows), 256, 0, stream>>>(b, p.cut);
    });
  });
}

int launch_distill_backward(const LogitsLaunch& a, hipStream_t stream) {
  const Plan p = plan_backward(a);
  return by_rows(a, [&](const LogitsLaunch& b) {
    by_shape(b.z_bf16, p.shape, [&](auto type, auto shape) {
      using T = decltype(type);
      constexpr int NT = decltype(shape)::threads, U = decltype(shape)::unroll;
      distill_backward_kernel<T, NT, U><<<grid_of(b, p), NT, 0, stream>>>(b, p.cut);
    });
  });
}

int launch_distill_step(const LogitsLaunch& a, hipStream_t stream) {
  const int64_t whole = a.vocab / (a.z_bf16 ? 8 : 4);  // vectors
  // A workgroup a row, or the forward and the gradient one after the other, which
  // cut rows for few of them. Both sides, us a call with 64 alternatives:
  //            rows:   1            32           64           96
  //   131072 bf16    18.7 / 20.8  20.5 / 23.2  20.7 / 26.4  21.4 / 30.5
  //   131072 f32     23.7 / 21.8  25.2 / 28.1  25.6 / 31.2  28.3 / 42.1
  //   151936 bf16    23.3 / 21.2  25.7 / 25.8  26.9 / 29.8  27.5 / 33.5
  //   230001 bf16    34.1 / 26.0  37.2 / 32.2  37.9 / 37.9  38.8 / 44.0
  //   200001 f32     34.3 / 23.4  37.6 / 28.8  40.2 / 40.2  46.5 / 56.2
  //   300001 bf16    40.9 / 23.1  44.7 / 25.7  46.2 / 37.6  48.2 / 45.4
  const int64_t from = a.vocab <= 131072 ? 1 : a.vocab <= 262144 ? 64 : 128;
  if (a.rows >= from)
    return by_rows(a, [&](const LogitsLaunch& b) {
      const auto with = [&](auto type) {
        using T = decltype(type);
        const unsigned grid = static_cast<unsigned>(b.rows);
        if (whole <= 1024) distill_step_kernel<T, 256, 4, false><<<grid, 256, 0, stream>>>(b);
        else if (whole <= 4096) distill_step_kernel<T, 256, 16, false><<<grid, 256, 0, stream>>>(b);
        else if (whole <= 8192) distill_step_kernel<T, 512, 16, false><<<grid, 512, 0, stream>>>(b);
        else if (whole <= 16384) distill_step_kernel<T, 1024, 16, false><<<grid, 1024, 0, stream>>>(b);
        else distill_step_kernel<T, 1024, 16, true><<<grid, 1024, 0, stream>>>(b);
      };
      if (b.z_bf16) with(uint16_t());
      else with(float());
    });
  if (launch_distill(a, stream) != 0) return -1;
  LogitsLaunch b = a;
  b.in_lse = a.lse;
  b.in_lse_tail = a.lse_tail;
  return launch_distill_backward(b, stream);
}

}  // namespace nvfp4

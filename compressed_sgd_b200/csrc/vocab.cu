// Losses over vocabulary rows: log probabilities of given tokens with the row's entropy and its most
// likely tokens, and distillation from a teacher's (index, value) list, each with the gradient of the
// logits in the same call or as a pass of its own.
//
// With z = x * it (it = 1 / temperature), c = it * log2(e) and any reference m, here at most 6.4 / c below the largest
// entry:
//   S = sum 2^((x - m) c),  T = sum 2^((x - m) c) (x - m) c,  p = 2^((x - m) c - log2 S),
//   entropy = ln2 (log2 S - T / S),  log p_t = (x_t - m) it - ln S,
// so one pass over a row gives everything but the gradient, and the gradient of either loss is p (A + B
// log2 p) per entry plus a few entries of the row's list, which are computed apart.
//
// What bounds them: a read of the logits (and a write of the gradient) at 6.5 TB/s, and next to it the
// exponential unit: one 2^x per entry and pass at 16 a clock and SM is 0.7 of the time that the bytes of
// 16-bit logits take. So the inner loops are counted in instructions: 6.6 per entry for the whole of a score with
// entropy (1184 x 85000 bf16), of which one is the exponential.
//
// Two kernels: voc_stream_kernel (losses, with or without the gradient, alternatives) and
// voc_backward_kernel (the gradient from saved statistics).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <type_traits>

#include "common.cuh"

namespace gs {
namespace {

namespace cg = cooperative_groups;

constexpr int kVocThreads = 256;
constexpr int kVocWarps = kVocThreads / 32;
constexpr int kUnroll = 4;                        // vectors of 16 bytes per lane and chunk
constexpr int kChunk = 32 * kUnroll;              // vectors per chunk
constexpr int kChunkLog = 7;
static_assert(kChunk == 1 << kChunkLog && kUnroll == 4, "");
constexpr int kStages = 3;                        // chunks per warp in the backward kernel's rings
constexpr int kCand = 2048;                       // candidates for a row's alternatives

constexpr float kLowest = -3.402823466e38f;       // the maximum of a row that holds nothing but -inf
constexpr float kFarBits = 1.0e4f;                // 2^-10^4 = 0: where a sum weighs by the exponent it is
                                                  // clamped here, so that -inf logits add 0
constexpr float kNearBits = 1048576.0f;           // references m with |m c| up to 2^20: exponents fma(x, c, -fl(m c)), which at
                                                  // m itself is the rounding of fl(m c), at most 2^-5. Beyond: (x - m) c

enum { kLogprob = 0, kRenorm = 1, kTail = 2 };    // what is computed
enum { kForward = 0, kFused = 1, kBackward = 2 }; // loss; loss and gradient; gradient from saved statistics

struct VocArgs {
  const void* logits;
  void* dlogits;
  int64_t stride, dstride;       // elements
  int32_t rows, vocab, split;    // split = CTAs per row
  int32_t slice;                 // vectors of a CTA's slice in shared memory
  uint32_t inv_split;            // ceil(2^32 / split)
  int32_t k;                     // list length: alternatives wanted (forward), given (backward), or the teacher's
  int32_t val_dtype;
  float it, c, c_lo;             // c + c_lo = it log2(e)
  float fine;                    // ln2 c_lo / c
  double inv_c;                  // 1 / c
  const int32_t* targets;
  const int32_t* list_idx;       // teacher's list, or the alternatives of the backward pass
  const void* list_val;          // teacher's values, or the gradient of the alternatives
  const float* stats_in;
  const float* entropy_in;
  const float* weight;           // gradient of logprob / of the loss, per row
  const float* weight_entropy;
  float* out;                    // logprob / loss
  float* entropy;
  float* stats;
  int32_t* top_idx;
  float* top_val;
  int32_t* d_status;
};

// ---- element types ------------------------------------------------------------------------

template <class T> struct Elem;
template <> struct Elem<float> {
  static constexpr int N = 4;
  using Max = float;                              // a running maximum, NaN passed over
  static __device__ __forceinline__ Max least() { return -INFINITY; }
  static __device__ __forceinline__ void rise(Max& m, const uint4& v) {
    m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v.x)), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ float top(const Max& m) { return m; }
  static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }   // -inf
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  // Largest entry of n vectors, NaN passed over (-inf or NaN if there is nothing else).
  template <int NV> static __device__ __forceinline__ float high(const uint4* v) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[u].x)), __uint_as_float(v[u].y)),
                fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
    return m;
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  using Max = __nv_bfloat162;
  static __device__ __forceinline__ Max least() { return as2(0xff80ff80u); }
  static __device__ __forceinline__ void rise(Max& m, const uint4& v) {
    m = __hmax2(__hmax2(m, as2(v.x)), __hmax2(__hmax2(as2(v.y), as2(v.z)), as2(v.w)));
  }
  static __device__ __forceinline__ float top(const Max& m) { return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y)); }
  static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }   // -inf
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
  template <int NV> static __device__ __forceinline__ float high(const uint4* v) {
    __nv_bfloat162 m = as2(v[0].x);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (u) m = __hmax2(m, as2(v[u].x));
      m = __hmax2(m, as2(v[u].y));
      m = __hmax2(m, as2(v[u].z));
      m = __hmax2(m, as2(v[u].w));
    }
    return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
  }
  static __device__ __forceinline__ __nv_bfloat162 as2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Elem<__half> {
  static constexpr int N = 8;
  using Max = __half2;
  static __device__ __forceinline__ Max least() { return as2(0xfc00fc00u); }
  static __device__ __forceinline__ void rise(Max& m, const uint4& v) {
    m = __hmax2(__hmax2(m, as2(v.x)), __hmax2(__hmax2(as2(v.y), as2(v.z)), as2(v.w)));
  }
  static __device__ __forceinline__ float top(const Max& m) { return fmaxf(__half2float(m.x), __half2float(m.y)); }
  static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u); }   // -inf
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
  template <int NV> static __device__ __forceinline__ float high(const uint4* v) {
    __half2 m = as2(v[0].x);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (u) m = __hmax2(m, as2(v[u].x));
      m = __hmax2(m, as2(v[u].y));
      m = __hmax2(m, as2(v[u].z));
      m = __hmax2(m, as2(v[u].w));
    }
    return fmaxf(__half2float(m.x), __half2float(m.y));
  }
  static __device__ __forceinline__ __half2 as2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float list_value(const void* p, int32_t dtype, int64_t i) {
  if (dtype == GSPARSE_F32) return static_cast<const float*>(p)[i];
  if (dtype == GSPARSE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// ---- arithmetic ---------------------------------------------------------------------------

// Two fp32 lanes in one instruction.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f2 v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// 2^x by the hardware's approximation (about 2 units in the last place; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Order of the alternatives: larger key = larger value, -0 = +0, NaN above +inf.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;      // order_key(-inf): never an alternative

// ---- block-wide reductions, in a fixed order ------------------------------------------------

// Largest of the warp's values, NaN passed over.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// One reduction's partial results. Every reduction of the kernel has its own, so that one barrier
// each is enough.
struct PartMax { float w[kVocWarps]; };
struct PartSum { double a[kVocWarps], b[kVocWarps]; };

// Maximum over the block, to every thread.
__device__ __forceinline__ float block_max(float v, PartMax& p) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) p.w[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float m = p.w[0];
  for (int w = 1; w < nw; ++w) m = fmaxf(m, p.w[w]);
  return m;
}
// Two sums over the block: put, a barrier, and any thread may get.
__device__ __forceinline__ void sum_put(double x, double y, PartSum& p) {
  x = warp_sum(x);
  y = warp_sum(y);
  if ((threadIdx.x & 31) == 0) {
    p.a[threadIdx.x >> 5] = x;
    p.b[threadIdx.x >> 5] = y;
  }
}
__device__ __forceinline__ void sum_get(double& x, double& y, const PartSum& p) {
  const int nw = blockDim.x >> 5;
  x = p.a[0];
  y = p.b[0];
  for (int w = 1; w < nw; ++w) {
    x += p.a[w];
    y += p.b[w];
  }
}
// Count over the block, to every thread; the barriers at both ends let the array be used again.
__device__ __forceinline__ int block_count(int v, int* part) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  int n = 0;
  for (int w = 0; w < nw; ++w) n += part[w];
  return n;
}

// 2^x for a small x to 64 bits' accuracy without the library's long route.
__device__ __forceinline__ double exp2_small(double x) {
  if (fabs(x) > 1.0e-4) return exp2(x);
  const double y = x * 0.6931471805599453;
  return 1.0 + y * (1.0 + y * (0.5 + y * (1.0 / 6.0)));   // next term below 1e-18
}

// ---- a row and its parts --------------------------------------------------------------------

// A row of V entries from `x`: `head` entries up to the first 16-byte boundary, `nv` whole vectors,
// and the tail. CTA `part` of `split` takes vectors [v0, v1); the head belongs to the first CTA, the
// tail to the last. Nothing outside the row is read.
template <class T>
struct Row {
  const T* x;
  int V, head, nv, v0, v1;
  bool first, last;
  // inv: ceil(2^32 / split), for n / split = (n inv) >> 32, exact for n split < 2^32.
  __device__ __forceinline__ Row(const T* p, int vocab, int part, int split, uint32_t inv) : x(p), V(vocab) {
    constexpr int N = Elem<T>::N;
    head = (int)(((16u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
    if (head > V) head = V;
    nv = (V - head) / N;
    v0 = split == 1 ? 0 : (int)__umulhi((uint32_t)nv * (uint32_t)part, inv);
    v1 = split == 1 ? nv : (int)__umulhi((uint32_t)nv * (uint32_t)(part + 1), inv);
    first = part == 0;
    last = part == split - 1;
  }
  __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(x + head); }
  __device__ __forceinline__ int tail0() const { return head + nv * Elem<T>::N; }
  // Element of the head or tail that thread t takes, or -1.
  __device__ __forceinline__ int edge(int t) const {
    if (first && t < head) return t;
    const int e = tail0() + (t - 32);             // the second warp takes the tail
    if (last && t >= 32 && e < V) return e;
    return -1;
  }
  __device__ __forceinline__ bool owns(int e) const {
    if (e < head) return first;
    const int v = (e - head) / Elem<T>::N;
    return v >= nv ? last : v >= v0 && v < v1;
  }
};

// ---- list of a row ------------------------------------------------------------------------------

struct List {              // in dynamic shared memory, for n entries
  double* q;               // the teacher's probability
  int32_t* idx;            // -1: absent
  float* x;                // the row's entry there
  float* v;                // the teacher's value, or the incoming gradient of the entry
  uint32_t* table;         // which indices are in the list: index + 1, open addressing, at most half full
  int slots;
  __host__ __device__ __forceinline__ static int table_slots(int n) {
    int t = 64;
    while (t < 2 * n) t *= 2;
    return t;
  }
  __host__ __device__ __forceinline__ static size_t bytes(int n) {
    return (size_t)round_up(n, 4) * 20 + (size_t)table_slots(n) * 4;
  }
  __device__ __forceinline__ void carve(void* at, int n) {
    const int m = (int)round_up(n, 4);
    q = static_cast<double*>(at);
    idx = reinterpret_cast<int32_t*>(q + m);
    x = reinterpret_cast<float*>(idx + m);
    v = x + m;
    table = reinterpret_cast<uint32_t*>(v + m);
    slots = table_slots(n);
  }
  // Enters index e; true if it was there.
  __device__ __forceinline__ bool add(int e) const {
    const uint32_t key = (uint32_t)e + 1u;
    uint32_t s = (key * 2654435761u) >> 16;
    for (int n = 0; n < slots; ++n, ++s) {
      const uint32_t old = atomicCAS(&table[s & (slots - 1)], 0u, key);
      if (old == 0u) return false;
      if (old == key) return true;
    }
    return false;
  }
};

// ---- most likely tokens ---------------------------------------------------------------------------

struct TopShared {
  unsigned long long cand[kCand];   // key << 32 | ~index: larger = earlier in the output
  int count;
};

__device__ __forceinline__ unsigned long long cand_of(uint32_t key, int e) {
  return ((unsigned long long)key << 32) | (uint32_t)~e;
}
__device__ __forceinline__ void cand_push(TopShared& t, uint32_t key, int e) {
  const int n = atomicAdd(&t.count, 1);
  if (n < kCand) t.cand[n] = cand_of(key, e);
}

// Entries of the whole row with key >= t (the CTA reads all of it).
template <class T>
__device__ int count_ge(const Row<T>& row, uint32_t t, int* sh) {
  int n = 0;
  const uint4* p = row.vec();
  for (int i = threadIdx.x; i < row.nv; i += blockDim.x) {
    float x[Elem<T>::N];
    Elem<T>::unpack(__ldcg(p + i), x);
#pragma unroll
    for (int j = 0; j < Elem<T>::N; ++j) n += order_key(x[j]) >= t;
  }
  for (int e = threadIdx.x; e < row.head; e += blockDim.x) n += order_key(Elem<T>::to(row.x[e])) >= t;
  for (int e = row.tail0() + threadIdx.x; e < row.V; e += blockDim.x) n += order_key(Elem<T>::to(row.x[e])) >= t;
  return block_count(n, sh);
}

// The alternatives of rows that the candidate store cannot hold (many equal entries, rows with
// NaN): bisection on the key for the k-th largest, then everything above it, then the entries equal
// to it from the lowest index on. Every step reads the row, which L2 holds by now.
template <class T>
__device__ __noinline__ void exact_top(const Row<T>& row, int k, uint32_t lower, TopShared& top, int* sh) {
  constexpr uint32_t kLeast = kKeyNegInf + 1;
  uint32_t lo = lower > kLeast ? lower : kLeast;      // at least k at or above lo, or lo = kLeast
  int above_lo = count_ge(row, lo, sh);
  bool ties = false;
  int above = 0;
  if (above_lo > kCand) {
    if (lo != 0xffffffffu) {
      above = count_ge(row, lo + 1, sh);
      if (above < k) {
        ties = true;
      } else {
        uint32_t l = lo + 1, h = 0xffffffffu;         // count(l) >= k throughout
        int nl = above;
        while (l < h && nl > kCand) {
          const uint32_t mid = l + (h - l + 1) / 2;
          const int n = count_ge(row, mid, sh);
          if (n >= k) {
            l = mid;
            nl = n;
          } else {
            h = mid - 1;
            above = n;
          }
        }
        lo = l;
        if (nl > kCand) {                             // l = h: the k-th key itself
          ties = true;
          above = lo == 0xffffffffu ? 0 : count_ge(row, lo + 1, sh);
        }
      }
    } else {
      ties = true;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) top.count = 0;
  __syncthreads();
  const uint32_t from = ties ? lo + 1 : lo;           // collected whole (lo = 0xffffffff: none)
  if (!(ties && lo == 0xffffffffu)) {
    for (int e = threadIdx.x; e < row.V; e += blockDim.x) {
      const uint32_t key = order_key(Elem<T>::to(row.x[e]));
      if (key >= from) cand_push(top, key, e);
    }
  }
  __syncthreads();
  if (!ties) return;
  int need = k - above, found = 0;
  for (int base = 0; base < row.V && found < need; base += blockDim.x) {
    const int e = base + threadIdx.x;
    const bool hit = e < row.V && order_key(Elem<T>::to(row.x[e])) == lo;
    const uint32_t b = __ballot_sync(kFull, hit);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = __popc(b);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
      if (w < (int)(threadIdx.x >> 5)) before += sh[w];
      all += sh[w];
    }
    before += __popc(b & lanemask_lt());
    if (hit && found + before < need) cand_push(top, lo, e);
    found += all;
  }
  __syncthreads();
}

// ---- a warp's chunks in shared memory ------------------------------------------------------------------

// Warp w of nw takes chunks w, w + nw, ... of its CTA's slice, each kChunk vectors (2 KB), copied
// by bulk asynchronous copies into a ring of its own: no warp waits for another, and kStages
// chunks per warp are on their way whatever the registers hold.
struct Ring {
  uint4* slots;
  uint64_t* bars;
  const uint4* from;      // the slice
  int own, n;             // vectors of the slice, chunks of this warp
  int warp, nw;
  uint32_t phase;         // parity of the next fill of each slot
  bool ok;
  __device__ __forceinline__ void init(uint4* s, uint64_t* b, const uint4* src, int vectors) {
    warp = threadIdx.x >> 5;
    nw = blockDim.x >> 5;
    slots = s + warp * kStages * kChunk;
    bars = b + warp * kStages;
    from = src;
    own = vectors;
    const int chunks = (vectors + kChunk - 1) / kChunk;
    n = chunks > warp ? (chunks - warp + nw - 1) / nw : 0;
    phase = 0;
    ok = true;
    if ((threadIdx.x & 31) == 0) {
      for (int q = 0; q < kStages; ++q) mbar_init(&bars[q], 1);
      fence_mbarrier_init();
    }
    __syncwarp();
  }
  __device__ __forceinline__ int first(int k) const { return (warp + nw * k) * kChunk; }   // vector of the slice
  __device__ __forceinline__ uint4* at(int k) const { return slots + (k % kStages) * kChunk; }
  // Requests chunk k (the slot's last readers have passed a __syncwarp).
  __device__ __forceinline__ void issue(int k) const {
    if ((threadIdx.x & 31) == 0) {
      const int o = first(k);
      const uint32_t bytes = 16u * (uint32_t)min(kChunk, own - o);
      mbar_arrive_expect_tx(&bars[k % kStages], bytes);
      bulk_load(at(k), from + o, bytes, &bars[k % kStages]);
    }
  }
  // Waits for the requested chunk k. A wait that runs out ends all later ones: the call reports it and
  // goes on with what the slot holds.
  __device__ __forceinline__ void wait(int k, int32_t* d_status) {
    const int q = k % kStages;
    if (ok && !mbar_wait_bounded(&bars[q], (phase >> q) & 1u)) {
      ok = false;
      raise(d_status, GSPARSE_DERR_TIMEOUT);
    }
    phase ^= 1u << q;
  }
  // No copy may land after the CTA is gone.
  __device__ __forceinline__ void drain() const {
    if (ok) return;
    for (int q = 0; q < kStages; ++q)
      for (uint32_t p = 0; p < 2; ++p) mbar_wait_bounded(&bars[q], p);
  }
};

// ---- gradient from saved statistics ----------------------------------------------------------------

constexpr int kHitWords = 16;

// The factors of the dense gradient for p = 2^((x - ref) c) / S, g = p (A + Bl log2 p). A reference beyond kNearBits
// (away) leaves the difference to the entries and k = E.
// With S = 2^E s, 1 <= s < 2, p = 2^(x c - k) f for k = fl(fl(ref c) + E) and f = 2^(k - E - ref c) / s: no
// logarithm, and no rounding of k is left in p.
template <class Out>
__device__ __forceinline__ void dense_factors(Out& R, float ref, double S, double A, double Bl, const VocArgs& a) {
  R.ref = ref;
  R.away = !(fabsf(ref) * a.c <= kNearBits);
  if (S == 0.0) {                                 // -inf alone, and entries that the list writes
    R.k = R.A = R.Bl = 0.0f;
    R.away = 0;
    return;
  }
  int E;
  const double s = 2.0 * frexp(S, &E);
  E -= 1;
  const float k = ref * a.c + (float)E;
  const double off = R.away ? 0.0 : (double)k - (double)E - (double)ref * (double)a.c;
  const double f = exp2_small(off) / s;
  R.k = R.away ? (float)E : k;
  R.A = (float)(f * (A + (Bl != 0.0 ? Bl * (off - (double)log2f((float)s)) : 0.0)));
  R.Bl = (float)(f * Bl);
}

// What one thread works out for all: 64-bit arithmetic by every thread would cost more than the row.
struct RowShared {
  PartMax max_list;
  PartSum sum_list;
  int repeats;         // an index stands in the list twice
  double Q, rho;       // mass of the list and what it leaves; kLogprob: sum of the gradients and of their sizes
  double list_max, list_sum;
  float ref, ref_row;
  double S_row;
  float k, A, Bl, A_list;
  int away;
  int empty;           // no entry in the teacher's list
};

// Dynamic shared memory: the warps' rings, then the list.
__host__ __device__ __forceinline__ size_t ring_bytes(int threads) { return (size_t)threads / 32 * kStages * kChunk * 16; }

// C CTAs take a row, each a slice, with nothing to tell each other. One read and one write per entry:
// 4096 x 32000 fp32 in 157 us, 6.69 TB/s; through registers, without the rings, 187 us.
template <class T, int OP>
__global__ void __launch_bounds__(kVocThreads, 4) voc_backward_kernel(const __grid_constant__ VocArgs a) {
  constexpr int N = Elem<T>::N, U = kUnroll;
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ RowShared R;
  __shared__ uint64_t bars[kVocWarps * kStages];

  const int C = a.split, r = C == 1 ? (int)blockIdx.x : (int)__umulhi(blockIdx.x, a.inv_split), part = (int)blockIdx.x - r * C;
  const int tid = threadIdx.x, lane = tid & 31, B = blockDim.x;
  const Row<T> row(static_cast<const T*>(a.logits) + (int64_t)r * a.stride, a.vocab, part, C, a.inv_split);
  const int own = row.v1 - row.v0, edge = row.edge(tid);
  Ring ring;
  ring.init(dyn, bars, row.vec() + row.v0, own);
  pdl_begin();

  // -- the row's list ---------------------------------------------------------------------------
  float w = a.weight ? a.weight[r] : 0.0f;        // gradient weights of the row
  const float w_h = OP == kLogprob && a.weight_entropy ? a.weight_entropy[r] : 0.0f;
  float x_edge = 0.0f;
  if (edge >= 0) x_edge = Elem<T>::to(row.x[edge]);
  int target = -1;
  if (OP == kLogprob && a.targets) {
    target = a.targets[r];
    if (target < -1 || target >= a.vocab) {
      if (tid == 0 && part == 0) raise(a.d_status, GSPARSE_DERR_INDEX_RANGE);
      target = -1;
    }
  }
  if (OP == kLogprob && target < 0) w = 0.0f;
  // nothing is read of a row without weights (where the list has none of its own)
  const bool early = OP == kLogprob || w != 0.0f;
  if (early)
    for (int q = 0; q < min(kStages, ring.n); ++q) ring.issue(q);
  const int nl = OP == kLogprob ? a.k + 1 : a.k;
  List L;
  L.carve(reinterpret_cast<char*>(dyn) + ring_bytes(B), nl);
  for (int i = tid; i < L.slots; i += B) L.table[i] = 0;
  if (tid == 0) R.repeats = 0;
  float vmax = -INFINITY;
  for (int j = tid; j < nl; j += B) {
    int e;
    float v;
    if (OP == kLogprob) {
      e = j == 0 ? target : a.list_idx[(int64_t)r * a.k + j - 1];
      v = j == 0 ? w : static_cast<const float*>(a.list_val)[(int64_t)r * a.k + j - 1];
    } else {
      e = a.list_idx[(int64_t)r * a.k + j];
      v = list_value(a.list_val, a.val_dtype, (int64_t)r * a.k + j);
    }
    if (e < -1 || e >= a.vocab) {
      if (part == 0) raise(a.d_status, GSPARSE_DERR_INDEX_RANGE);
      e = -1;
    }
    L.idx[j] = e;
    L.x[j] = e >= 0 && row.owns(e) ? Elem<T>::to(row.x[e]) : 0.0f;
    L.v[j] = v;
    if (e >= 0) vmax = fmaxf(vmax, v);
  }
  float list_max = 0.0f;
  if (OP == kRenorm) list_max = fmaxf(block_max(vmax, R.max_list), kLowest);
  else __syncthreads();
  // sum of the probabilities (of the renormalised list: not yet divided) and how many; of the incoming gradients and
  // their sizes
  double sum = 0.0, size = 0.0;
  for (int j = tid; j < nl; j += B) {
    const int e = L.idx[j];
    if (e < 0) continue;
    if (OP == kLogprob) {
      if (j > 0) sum += (double)L.v[j];
      size += fabs((double)L.v[j]);
    } else {
      const double q = exp(OP == kRenorm ? ((double)L.v[j] - (double)list_max) * (double)a.it : (double)L.v[j]);
      L.q[j] = q;
      sum += q;
      size += 1.0;
    }
    if (L.add(e)) R.repeats = 1;
  }
  sum_put(sum, size, R.sum_list);
  __syncthreads();

  // -- the dense gradient's factors ----------------------------------------------------------------
  if (tid == 0) {
    sum_get(sum, size, R.sum_list);
    R.Q = sum;
    R.rho = size;
    R.empty = size == 0.0;
    R.list_sum = sum;
    if (OP == kRenorm) R.Q = sum == 0.0 ? 0.0 : sum == sum ? 1.0 : sum;
    if (OP == kTail) R.rho = sum == sum ? fmax(1.0 - sum, 0.0) : sum;
    const float* st = a.stats_in + (int64_t)r * (OP == kTail ? 4 : 2);
    float ref = fmaxf(st[0], kLowest);
    double S = (double)st[1];
    R.ref_row = ref;
    R.S_row = S;
    if (OP == kTail) {
      ref = fmaxf(st[2], kLowest);
      S = (double)st[3];
      if (S == 0.0) R.rho = 0.0;                  // no entry is left for the rest
    }
    const double it = (double)a.it;
    double A, Bl = 0.0;
    if (OP == kLogprob) {
      A = -it * ((double)w + R.Q + (w_h != 0.0f ? (double)w_h * (double)a.entropy_in[r] : 0.0));
      Bl = -it * (double)w_h * 0.6931471805599453;
      R.A_list = (float)A;
    } else if (OP == kRenorm) {
      A = it * (double)w * R.Q;
      R.A_list = (float)A;
    } else {
      const double Rr = S == 0.0 ? 0.0
                        : S / R.S_row * (ref == R.ref_row ? 1.0 : exp(((double)ref - (double)R.ref_row) * it));
      A = it * (double)w * ((R.Q + R.rho) * Rr - R.rho);
      R.A_list = (float)(it * (double)w * (R.Q + R.rho));
    }
    dense_factors(R, ref, S, A, Bl, a);
  }
  __syncthreads();

  // -- gradient ------------------------------------------------------------------------------------
  const float kf = R.k, A = R.A, Bl = R.Bl, ref = R.ref;
  const bool nothing = R.S_row == 0.0;            // nothing but -inf: no distribution, no gradient
  // no weight: zeros, whatever the row holds
  const bool none = nothing || (OP == kLogprob ? w_h == 0.0f && R.rho == 0.0 : w == 0.0f || R.empty);
  const bool away = R.away;
  T* dx = static_cast<T*>(a.dlogits) + (int64_t)r * a.dstride;
  const f2 c2 = pair(a.c, a.c), nk = pair(-kf, -kf), A2 = pair(A, A), B2 = pair(Bl, Bl);
  auto grad = [&](uint4 v, auto far) {             // far: the difference first
    float x[N];
    Elem<T>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float q0, q1;
      f2 q, g = A2;
      if constexpr (far.value) {
        q0 = max_nan((x[i] - ref) * a.c, -kFarBits) - kf;
        q1 = max_nan((x[i + 1] - ref) * a.c, -kFarBits) - kf;
      } else {
        q = fma2(pair(x[i], x[i + 1]), c2, nk);
        unpair(q, &q0, &q1);
      }
      if (OP == kLogprob && Bl != 0.0f) g = fma2(pair(max_nan(q0, -kFarBits), max_nan(q1, -kFarBits)), B2, A2);
      unpair(mul2(pair(ex2(q0), ex2(q1)), g), &x[i], &x[i + 1]);
    }
    return Elem<T>::pack(x);
  };
  auto grad_one = [&](float x) {
    const float q = away ? max_nan((x - ref) * a.c, -kFarBits) - kf : fmaf(x, a.c, -kf);
    return Elem<T>::from(ex2(q) * (Bl != 0.0f ? fmaf(max_nan(q, -kFarBits), Bl, A) : A));
  };
  const int e0 = row.head + row.v0 * N, e1 = row.head + row.v1 * N;
  const bool in_step = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(row.x)) & 15u) == 0;
  uint4* dvec = reinterpret_cast<uint4*>(dx + row.head) + row.v0;
  if (early && (none || !in_step))
    for (int q = 0; q < min(kStages, ring.n); ++q) ring.wait(q, a.d_status);
  if (none) {
    if (in_step) {
      for (int i = tid; i < own; i += B) __stcs(dvec + i, make_uint4(0, 0, 0, 0));
    } else {
      for (int e = e0 + tid; e < e1; e += B) dx[e] = Elem<T>::from(0.0f);
    }
    if (edge >= 0) dx[edge] = Elem<T>::from(0.0f);
    ring.drain();
    return;
  }
  auto chunks = [&](auto far) {
    for (int q = 0; q < ring.n; ++q) {
      ring.wait(q, a.d_status);
      const uint4* at = ring.at(q);
      uint4* to = dvec + ring.first(q);
      const int left = own - ring.first(q);
      if (left >= kChunk) {
#pragma unroll
        for (int u = 0; u < U; ++u) __stcs(to + u * 32 + lane, grad(at[u * 32 + lane], far));
      } else {
        for (int u = lane; u < left; u += 32) __stcs(to + u, grad(at[u], far));
      }
      __syncwarp();
      if (q + kStages < ring.n) ring.issue(q + kStages);
    }
  };
  if (in_step) {
    if (away) chunks(std::true_type{});
    else chunks(std::false_type{});
  } else {                                        // rows that start at different offsets from 16 bytes
    for (int e = e0 + tid; e < e1; e += B) dx[e] = grad_one(Elem<T>::to(row.x[e]));
  }
  if (edge >= 0) dx[edge] = grad_one(x_edge);
  ring.drain();
  __syncthreads();
  // the list's entries, in 64 bits, over what the dense part wrote there
  const double per = OP == kRenorm ? -(double)w / R.list_sum : -(double)w;
  for (int j = tid; j < nl; j += B) {
    const int e = L.idx[j];
    if (e < 0 || !row.owns(e)) continue;
    double add = 0.0;
    bool mine = true;
    for (int i = R.repeats ? 0 : j; i < (R.repeats ? nl : j + 1); ++i) {
      if (L.idx[i] != e) continue;
      if (i < j) mine = false;
      if (OP == kLogprob) add += (double)L.v[i];
      else if (R.Q != 0.0) add += per * L.q[i];
    }
    if (!mine) continue;
    const double z = ((double)L.x[j] - (double)R.ref_row) * (double)a.it, p = exp(z) / R.S_row;
    double g = p * (double)R.A_list + (double)a.it * add;
    if (OP == kLogprob && w_h != 0.0f && p != 0.0) g -= (double)a.it * (double)w_h * p * (z - log(R.S_row));
    dx[e] = Elem<T>::from((float)g);
  }
}

// ---- sums without a running maximum ---------------------------------------------------------------------

// Sums over a lane's entries of e = 2^q and e q. The reference is the largest entry m of the first chunk in which
// the warp finds one, near 0: q = fma(x, c, -rc), rc = fl(m c), the same for every entry; away from it: q = (x - m) c.
// (4000 x 85000 bf16, scores and with the gradient: ordinary rows 111 and 268 us, rows away from 0 124 and 369: their
// factors are worked out in 64 bits.)
// Entries above it are added as they are until a chunk takes the sums T beyond kShiftAt, which moves it. Saves half an
// instruction per entry against the running maximum. A chunk's entries are added up before they join s and t, so that a
// large entry swallows those of its own chunk at most. All but s and t is the warp's.
// NaN or +inf make the row NaN: nothing more is read of the warp's chunks.
enum { kNone = 0, kNear = 1, kAway = 2, kNan = 3 };   // what there is (parts of a row: up to kAway)
// An entry 6.4 bits above the reference moves it: T / S from a reference k bits below the row's largest entry has k
// roundings, and the entropy log S - T / S may be next to nothing. (No slower than 2^60: 4000 x 85000 bf16 118 us.)
constexpr float kShiftAt = 512.0f;

struct Sums {
  int kind;
  float ref;              // kNear: rc, kAway: m
  f2 s, t;
  bool gaps;              // -inf has been met (0 * -inf makes t NaN): exponents are clamped from there on
};

// Moves the reference to a chunk's largest entry over the warp, from kNone too.
__device__ __noinline__ Sums sums_move(Sums r, float top, float c) {
  const float rc = top * c;
  const bool near = fabsf(rc) <= kNearBits;
  float down = 0.0f;                              // from the new reference to the old one
  if (top == INFINITY) {
    r.kind = kNan;
  } else if (r.kind == kNone) {
    r.kind = near ? kNear : kAway;
    r.ref = near ? rc : top;
  } else if (r.kind == kNear && rc > r.ref) {
    down = near ? r.ref - rc : fmaf(-top, c, r.ref);
    r.kind = near ? kNear : kAway;
    r.ref = near ? rc : top;
  } else if (r.kind == kAway && top > r.ref) {
    down = (r.ref - top) * c;
    r.ref = top;
    if (near && down < -kFarBits) {               // nothing is left of what was there
      r.kind = kNear;
      r.ref = rc;
    }
  }
  if (down < 0.0f) {
    down = fmaxf(down, -kFarBits);
    const float f = ex2(down);
    r.t = mul2(fma2(r.s, pair(down, down), r.t), pair(f, f));
    r.s = mul2(r.s, pair(f, f));
  }
  return r;
}

// Adds NV vectors to the sums, unless a lane's T is then beyond kShiftAt or NaN; returns that T. FAST: references near 0, no
// -inf: entry by entry unpack, half a fused multiply-add, 2^q, half an addition, half a fused multiply-add. Else half
// an addition (the difference with a reference away from 0) and a maximum more.
template <class T, int NV, bool FAST>
__device__ __forceinline__ float sums_some(Sums& r, const uint4* v, float c) {
  constexpr int N = Elem<T>::N;
  const float m = r.kind == kAway ? r.ref : 0.0f, rc = r.kind == kAway ? 0.0f : r.ref;
  const f2 c2 = pair(c, c), nrc = FAST ? pair(-r.ref, -r.ref) : pair(-rc, -rc), nm = pair(-m, -m);
  f2 s = pair(0.0f, 0.0f), t = s;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    float x[N];
    Elem<T>::unpack(v[u], x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      f2 q = pair(x[i], x[i + 1]);
      if (!FAST) q = add2(q, nm);
      q = fma2(q, c2, nrc);
      float q0, q1;
      unpair(q, &q0, &q1);
      if (!FAST) {
        q0 = max_nan(q0, -kFarBits);
        q1 = max_nan(q1, -kFarBits);
        q = pair(q0, q1);
      }
      const f2 e = pair(ex2(q0), ex2(q1));
      s = add2(s, e);
      t = fma2(e, q, t);
    }
  }
  float t0, t1;
  unpair(t, &t0, &t1);
  t0 += t1;
  if (__all_sync(kFull, t0 < kShiftAt)) {
    r.s = add2(r.s, s);
    r.t = add2(r.t, t);
    return 0.0f;
  }
  return __any_sync(kFull, t0 != t0) ? NAN : kShiftAt;
}

// Adds a chunk; gaps: it may hold -inf.
template <class T, int NV>
__device__ __forceinline__ void sums_add(Sums& r, const uint4* v, const VocArgs& a, bool gaps = false) {
  if (r.kind == kNan) return;
  bool move = false;
  if (r.kind == kNone) {
    const float top = warp_max(Elem<T>::template high<NV>(v)), rc = top * a.c;
    if (fabsf(rc) <= kNearBits) {
      r.kind = kNear;
      r.ref = rc;
    } else {
      move = true;
      if (!(top > -INFINITY)) {                   // -inf alone, or NaN
        bool all = true;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          const uint32_t no = Elem<T>::nothing().x;
          all = all && v[u].x == no && v[u].y == no && v[u].z == no && v[u].w == no;
        }
        if (!__all_sync(kFull, all)) r.kind = kNan;
        return;
      }
    }
  }
  if (r.kind == kNear && !r.gaps && !gaps) {
    const float t = sums_some<T, NV, true>(r, v, a.c);
    if (t == 0.0f) return;
    move = t == t;
    r.gaps = !move;
  }
  while (true) {                                  // from a chunk's largest entry its T is below kShiftAt: at most twice
    if (move) r = sums_move(r, warp_max(Elem<T>::template high<NV>(v)), a.c);
    if (r.kind == kNan) return;
    const float t = sums_some<T, NV, false>(r, v, a.c);
    if (t == 0.0f) return;
    if (move || t != t) {
      r.kind = kNan;
      return;
    }
    move = true;
  }
}

// Reads a row's vector past L1. (Kept coherent: the gradient may take the logits' place.)
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Asynchronous 16-byte copies by each lane for itself.
__device__ __forceinline__ void copy_async(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// ---- a row per cluster, streamed -----------------------------------------------------------------------

// A cluster of C CTAs takes a row; W warps of a CTA stream its slice chunk by chunk (U vectors per lane) and
// one more warp reads the row's list, joins the partial sums and writes the results, in 64 bits where that
// is free. The warps meet once per row: each sends its partial sums to every CTA of the row that needs them.
// C = 1 when there are rows enough to fill the GPU and no gradient.
//
// Sums alone: the next chunk's loads are in registers while one is worked on, 64 KB a SM on their way. Measured on
// 4000 rows of 85000 bf16 (680 MB): 118 us, 5.8 TB/s, 0.88 of the measured copy bandwidth. A kernel that only
// reads takes 95 us with such loads and 109 to 120 us with cp.async rings of 64 to 192 KB a SM; this one with bulk
// or cp.async rings took 133 to 190 us.
//
// RES (with the gradient): the slice goes to shared memory and stays there between the sums and the gradient:
// 303 us, 4.5 TB/s, 0.69. Reading it again from L2 instead costs half as much traffic again between L2 and the
// SMs (322 us), and more than about 60 MB of rows in flight no longer stay in L2. What is left is the chain of
// a slice, about 9 us for 42 KB (loads 2, sums 3, join 1.5, gradient 2.5), of which four CTAs per SM hide two
// thirds. Rows that eight slices of 200 KB cannot hold are read twice.
constexpr int kRowWarps = 7;                      // streaming warps, at most
constexpr int kRowCtas = 4;                       // per SM
constexpr int kAhead = 2;                         // chunks per warp on their way to shared memory (RES)
constexpr int kParts = 8 * kRowWarps;             // partial sums of a row, at most

struct StreamShared {
  uint64_t listed, sums, factors, ready;          // the list's indices; all partial sums; the gradient's factors; that at the list's entries
  uint64_t gathered;                              // the row's entries at the list have been read
  uint64_t bounded, pushed;                       // alternatives: the CTAs' bounds are there; all candidates
  uint32_t bounds[8], tops[8], least[8];
  alignas(16) uint32_t reach[2][8];               // parts of each warp that reach three values, ten bits each
  int owners;
  int nan, scratch[kRowWarps + 1];
  float top_ref;
  double top_log_s;
  float4 part[kParts];                            // of each warp: reference, s, t, and as an int its kind
  int repeats;                                    // an index stands in the list twice
  uint32_t hit[kHitWords];                        // chunks of the slice that hold entries of the list (modulo)
  float w, w_h, x_target;
  int target;
  double Q, rho, list_max, list_sum;
  float list_high;                                // kTail: largest logit at the list's entries
  double list_exp;                                // and the sum of exp(z - its z) over them
  // the gradient's factors
  float k, A, Bl, ref;
  int away, none;
  int empty;                                      // no entry in the list
  float g_target;                                 // the gradient at the target
};

// Stores to and arrivals at another CTA of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, int q) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(q));
  return r;
}
// The store itself counts on the barrier there: a release over the cluster before an arrival costs the warp
// about 2000 cycles.
__device__ __forceinline__ void peer_send(float4* p, uint64_t* bar, int q, float4 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(peer(p, q)),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(peer(bar, q))
               : "memory");
}
__device__ __forceinline__ void peer_arrive(uint64_t* bar, int q) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer(bar, q)) : "memory");
}
// Waits, asleep, until the barrier's first phase is complete; false after kWaitCycles.
__device__ __forceinline__ bool peer_try_wait(uint64_t* bar) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0, 1000000;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar))
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool peer_wait_bounded(uint64_t* bar) {
  if (peer_try_wait(bar)) return true;
  const long long t0 = clock64();
  while (!peer_try_wait(bar))
    if (clock64() - t0 > kWaitCycles) return false;
  return true;
}

// Places for n candidates in the first CTA of the row (alone: the row has no other), and a candidate there.
__device__ __forceinline__ uint32_t peer_places(TopShared* top, int n, bool alone) {
  if (alone) return (uint32_t)atomicAdd(&top->count, n);
  uint32_t at;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(peer(&top->count, 0)), "r"(n) : "memory");
  return at;
}
__device__ __forceinline__ void peer_put(TopShared* top, uint32_t at, uint32_t key, int e, bool alone) {
  if (at >= kCand) return;
  if (alone) top->cand[at] = cand_of(key, e);
  else asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer(&top->cand[at], 0)), "l"(cand_of(key, e)) : "memory");
}

// Shared memory: RES: the slice; else a chunk per warp for those that hold entries of the list. Then the
// list; with the alternatives, the maxima and the candidates.
template <class T, int OP, int MODE, bool RES, bool TOP>
__global__ void __launch_bounds__((kRowWarps + 1) * 32, kRowCtas) voc_stream_kernel(const __grid_constant__ VocArgs a) {
  constexpr int N = Elem<T>::N, U = kUnroll;
  constexpr bool LIST = OP != kLogprob;
  constexpr bool GRAD = MODE == kFused;
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ StreamShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = (blockDim.x >> 5) - 1;
  const int C = a.split, r = C == 1 ? (int)blockIdx.x : (int)__umulhi(blockIdx.x, a.inv_split), part = (int)blockIdx.x - r * C;
  const Row<T> row(static_cast<const T*>(a.logits) + (int64_t)r * a.stride, a.vocab, part, C, a.inv_split);
  const int own = row.v1 - row.v0, step = W * kChunk;
  uint4* const buf = RES ? dyn : dyn + warp * kChunk;
  List L;
  if constexpr (LIST) L.carve(dyn + (RES ? a.slice : W * kChunk), a.k);
  // alternatives: parts of the slice that hold candidates (a part is what a lane reads at one place of its
  // chunks), and the candidates
  uint16_t* owners = reinterpret_cast<uint16_t*>(dyn + W * kChunk);
  TopShared& top = *reinterpret_cast<TopShared*>(owners + W * 128);

  if (threadIdx.x == 0) {
    mbar_init(&sh.listed, 1);
    mbar_init(&sh.factors, 1);
    mbar_init(&sh.gathered, 1);
    mbar_init(&sh.sums, C == 1 ? W : 1);
    mbar_init(&sh.ready, 1);
    if (TOP) {
      mbar_init(&sh.bounded, C);
      mbar_init(&sh.pushed, part == 0 ? C * W : 1);
      top.count = 0;
      sh.owners = 0;
    }
    fence_mbarrier_init();
    if (C > 1 && (GRAD || part == 0)) mbar_arrive_expect_tx(&sh.sums, 16u * (uint32_t)(C * W));
  }
  __syncthreads();
  // the CTAs meet without waiting; what is sent to another waits for its start
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  auto started = [&]() {
    if (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  };
  pdl_begin();
  const uint4* at = row.vec() + row.v0 + warp * kChunk + lane;
  uint4 nx[U];
  auto request = [&](int left) {                  // of the slice, from the chunk's first vector on
    if constexpr (RES) {                          // straight to its place
      uint4* to = buf + (own - left) + lane;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * 32 + lane < left) copy_async(to + u * 32, at + u * 32);
      copy_commit();
    } else if (left >= kChunk) {
#pragma unroll
      for (int u = 0; u < U; ++u) nx[u] = ld_row(at + u * 32);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * 32 + lane < left) nx[u] = ld_row(at + u * 32);
    }
    at += step;
  };
  if (warp < W)
    for (int q = 0; q < (RES ? kAhead : 1); ++q) request(own - warp * kChunk - q * step);
  // the first warp's lanes take the head and the tail, one entry each
  int edge = -1;
  if (warp == 0) {
    if (row.first && lane < row.head) edge = lane;
    else if (row.last && lane >= 8 && row.tail0() + lane - 8 < row.V) edge = row.tail0() + lane - 8;
  }
  float x_edge = -INFINITY;
  if (edge >= 0) x_edge = Elem<T>::to(row.x[edge]);
  bool ok = true;                                 // a wait that runs out ends all later ones
  auto wait = [&](uint64_t* bar) {
    if (ok && !peer_wait_bounded(bar)) {
      ok = false;
      raise(a.d_status, GSPARSE_DERR_TIMEOUT);
    }
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
  };

  // What others send here is waited for, so that a CTA may leave when it is done; if a wait has run out it
  // stays until the others have left.
  auto leave = [&]() {
    if (C > 1 && !__all_sync(kFull, ok)) cg::this_cluster().sync();
  };

  if (warp == W) {
    // -- the row's list ----------------------------------------------------------------------------
    float w = 0.0f, w_h = 0.0f;
    if (GRAD) {
      w = a.weight ? a.weight[r] : 0.0f;
      w_h = OP == kLogprob && a.weight_entropy ? a.weight_entropy[r] : 0.0f;
    }
    if (OP == kLogprob) {
      int target = a.targets ? a.targets[r] : -1;
      if (target < -1 || target >= a.vocab) {
        if (lane == 0 && part == 0) raise(a.d_status, GSPARSE_DERR_INDEX_RANGE);
        target = -1;
      }
      w = target >= 0 ? w : 0.0f;
      if (lane == 0) {
        sh.target = target;
        sh.x_target = target >= 0 ? Elem<T>::to(row.x[target]) : 0.0f;
        sh.w = w;
        sh.w_h = w_h;
      }
    }
    if constexpr (LIST) {
      if (GRAD || OP == kTail)
        for (int i = lane; i < L.slots; i += 32) L.table[i] = 0;
      if (lane < kHitWords) sh.hit[lane] = 0;
      float vmax = -INFINITY;
#pragma unroll 4
      for (int j = lane; j < a.k; j += 32) {
        const int64_t o = (int64_t)r * a.k + j;
        int e = a.list_idx[o];
        const float v = list_value(a.list_val, a.val_dtype, o);
        if (e < -1 || e >= a.vocab) {
          if (part == 0) raise(a.d_status, GSPARSE_DERR_INDEX_RANGE);
          e = -1;
        }
        L.idx[j] = e;
        L.v[j] = v;
        if (e >= 0) vmax = fmaxf(vmax, v);
      }
      __syncwarp();
      // which chunks hold entries of the list: what the tail's sums begin with
      auto mark = [&]() {
        bool repeats = false;
        for (int j = lane; j < a.k; j += 32) {
          const int e = L.idx[j];
          if (e < 0) continue;
          repeats |= L.add(e);
          const int at = e < row.head ? -1 : (e - row.head) / N - row.v0;   // vector of the slice
          if (at >= 0 && at < own) {
            const int c = at / kChunk;
            atomicOr(&sh.hit[(c >> 5) & (kHitWords - 1)], 1u << (c & 31));
          }
        }
        repeats = __any_sync(kFull, repeats);
        if (lane == 0) sh.repeats = repeats;
        arrive(&sh.listed);
      };
      if (OP == kTail) mark();
#pragma unroll 4
      for (int j = lane; j < a.k; j += 32) {
        const int e = L.idx[j];
        L.x[j] = e >= 0 ? Elem<T>::to(row.x[e]) : 0.0f;
      }
      arrive(&sh.gathered);
      if (OP != kTail && GRAD) mark();
      vmax = fmaxf(warp_max(vmax), kLowest);
      bool any = false;
      double sum = 0.0;
      for (int j = lane; j < a.k; j += 32) {
        const int e = L.idx[j];
        if (e < 0) continue;
        const double q = exp(OP == kRenorm ? ((double)L.v[j] - (double)vmax) * (double)a.it : (double)L.v[j]);
        L.q[j] = q;
        sum += q;
        any = true;
      }
      sum = warp_sum(sum);
      any = __any_sync(kFull, any);
      if (lane == 0) {
        sh.empty = !any;
        sh.w = w;
        sh.list_max = (double)vmax;
        sh.list_sum = sum;
        sh.Q = OP == kTail ? sum : sum == 0.0 ? 0.0 : sum == sum ? 1.0 : sum;
        sh.rho = OP == kTail ? (sum == sum ? fmax(1.0 - sum, 0.0) : sum) : 0.0;
      }
    }
    if constexpr (OP == kTail && GRAD) {
      // what the entries add to the row's sum, from the largest of them
      float high = -INFINITY;
      for (int j = lane; j < a.k; j += 32)
        if (L.idx[j] >= 0) high = fmaxf(high, L.x[j]);
      high = warp_max(high);
      double add = 0.0;
      __syncwarp();
      for (int j = lane; j < a.k; j += 32) {
        if (L.idx[j] < 0) continue;
        bool count = true;
        if (sh.repeats)
          for (int i = 0; i < j; ++i) count = count && L.idx[i] != L.idx[j];
        if (count && !(L.x[j] == -INFINITY)) add += exp(((double)L.x[j] - (double)high) * (double)a.it);
      }
      add = warp_sum(add);
      if (lane == 0) {
        sh.list_high = high;
        sh.list_exp = add;
      }
    }
    if (!LIST) arrive(&sh.gathered);
    __syncwarp();
    started();
    if (!GRAD && part != 0) return;

    // -- the row's results in 64 bits ------------------------------------------------------------------
    wait(&sh.sums);
    bool near = true;                             // the row's parts have references near 0, or are nothing beside those that have
    auto beside = [&](const float4& p, float rcm) { return __float_as_int(p.w) == kAway && !(p.x * a.c < rcm - 2.0f * kFarBits); };
    if constexpr (GRAD) {
      // What the gradient waits for, in fp32, the parts in a fixed order (by every warp for itself this took 1400
      // instructions per CTA)
      const int parts = C * W;
      const float4 p = lane < parts ? sh.part[lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      bool normal = __float_as_int(p.w) == kNear;
      float rcm = warp_max(normal ? p.x : -INFINITY);
      float4 p1 = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      if (parts > 32) {
        if (lane + 32 < parts) p1 = sh.part[lane + 32];
        normal |= __float_as_int(p1.w) == kNear;
        rcm = fmaxf(rcm, warp_max(__float_as_int(p1.w) == kNear ? p1.x : -INFINITY));
      }
      near = __any_sync(kFull, normal) && !__any_sync(kFull, beside(p, rcm) || (parts > 32 && beside(p1, rcm)));
      if (near) {
        float s = 0.0f, t = 0.0f;
        if (__float_as_int(p.w) == kNear) {
          const float d = fmaxf(p.x - rcm, -kFarBits), f = ex2(d);
          s = f * p.y;
          t = f * fmaf(d, p.y, p.z);
        }
        if (parts > 32 && __float_as_int(p1.w) == kNear) {
          const float d = fmaxf(p1.x - rcm, -kFarBits), f = ex2(d);
          s = fmaf(f, p1.y, s);
          t = fmaf(f, fmaf(d, p1.y, p1.z), t);
        }
        s = warp_sum(s);
        t = warp_sum(t);
        float Af, Bl = 0.0f, ent = 0.0f;
        if (OP == kLogprob && w_h != 0.0f) ent = 0.69314718f * (__log2f(s) - __fdividef(t, s));
        s = fmaf(a.fine, t, s);                     // c is rounded: to first order S + d ln2 T
        if (OP == kLogprob) {
          Af = -a.it * fmaf(w_h, ent, w);
          Bl = -a.it * w_h * 0.69314718f;
        } else if (OP == kRenorm) {
          Af = a.it * w * (float)sh.Q;
        } else {
          // the list's sum to the same reference; the share of the others
          const float d = (float)(((double)sh.list_high - (double)rcm * a.inv_c) * ((double)a.c + (double)a.c_lo));
          const float Q = (float)sh.Q, rho = (float)sh.rho;
          float R = 1.0f;
          if (!(sh.list_exp == 0.0)) {
            // (beyond 2^100 the others are nothing beside the list)
            R = d < 100.0f ? s / (s + (float)sh.list_exp * ex2(d)) : s * ex2(-d) / (float)sh.list_exp;
          }
          Af = a.it * w * ((Q + rho) * R - rho);
        }
        // p = 2^(x c - rcm) / s with s = 2^E m: 2^(x c - k) f, k = fl(rcm + E), f = 2^(k - E - rcm) / m
        const int E = (int)((__float_as_uint(s) >> 23) & 255u) - 127;
        const float m = s * __uint_as_float((uint32_t)(127 - E) << 23);
        const float kf = rcm + (float)E;
        const float off = (float)((double)kf - (double)E - (double)rcm), f = __fdividef(ex2(off), m);
        const float A = f * (Bl != 0.0f ? fmaf(Bl, off - __log2f(m), Af) : Af);
        Bl *= f;
        if (lane == 0) {
          sh.k = kf;
          sh.A = A;
          sh.Bl = Bl;
          sh.ref = 0.0f;
          sh.away = 0;
          sh.none = (w == 0.0f && w_h == 0.0f) || (LIST && sh.empty);
        }
        arrive(&sh.factors);
      }
    }
    float M = -INFINITY;                          // what the sums are taken from
    double Sd = 0.0, Td = 0.0;
    const int n_parts = C * W;
    for (int q = lane; q < n_parts; q += 32)
      if (__float_as_int(sh.part[q].w) == kNear) M = fmaxf(M, sh.part[q].x);
    M = warp_max(M);
    if constexpr (!GRAD) {
      bool other = false;
      for (int q = lane; q < n_parts; q += 32) other |= beside(sh.part[q], M);
      near = M > -INFINITY && !__any_sync(kFull, other);
    }
    if (near) {
      for (int q = lane; q < n_parts; q += 32) {
        const float4 p = sh.part[q];
        if (__float_as_int(p.w) != kNear) continue;
        const float off = fmaxf(p.x - M, -kFarBits), f = ex2(off);
        Sd += (double)f * (double)p.y;
        Td += (double)f * ((double)p.z + (double)off * (double)p.y);
      }
      Sd = warp_sum(Sd);
      Td = warp_sum(Td);
      const double rc = (double)M;
      M = (float)(rc * a.inv_c);
      const double off = rc - (double)M * (double)a.c, f = exp2_small(off);
      Td = f * (Td + off * Sd);
      Sd *= f;
    } else {
      // the parts' references in bits, exact in 64 bits; the largest, and an entry at or near it
      auto bits = [&](const float4& p) { return __float_as_int(p.w) == kAway ? (double)p.x * (double)a.c : (double)p.x; };
      double high = -INFINITY;
      M = -INFINITY;
      for (int q = lane; q < n_parts; q += 32) {
        const float4 p = sh.part[q];
        if (__float_as_int(p.w) == kNone || !(bits(p) > high)) continue;
        high = bits(p);
        M = __float_as_int(p.w) == kAway ? p.x : (float)(high * a.inv_c);
      }
      double most = high;
      for (int d = 16; d > 0; d >>= 1) most = fmax(most, __shfl_xor_sync(kFull, most, d));
      M = warp_max(high == most ? M : -INFINITY);
      for (int q = lane; q < n_parts; q += 32) {
        const float4 p = sh.part[q];
        if (__float_as_int(p.w) == kNone) continue;
        const double off = bits(p) - (double)M * (double)a.c, s = (double)p.y, t = (double)p.z;
        // (a part that is nothing beside the others still brings its NaN)
        const double f = off < -2.0 * kFarBits ? 0.0 : exp2_small(off);
        Sd += f * s;
        Td += f == 0.0 ? f * s : f * (t + off * s);
      }
      Sd = warp_sum(Sd);
      Td = warp_sum(Td);
    }
    const float ref = fmaxf(M, kLowest);
    // c is rounded: to first order 2^(q (1 + d)) = 2^q (1 + d ln2 q), with the sum of 2^q q at hand. The entropy takes S
    // and T as they are: at a temperature off by d it is off by d times the variance of z, with S alone corrected by d times
    // the square of z's mean.
    const double S_raw = Sd;
    Sd += (double)a.fine * Td;
    float ref_row = ref;
    double S_row = Sd, loss = 0.0, rho = 0.0, Q = 0.0;
    if constexpr (LIST) {
      Q = sh.Q;
      rho = sh.rho;
      if (OP == kTail) {                          // the list's entries join the others
        float high = -INFINITY;
        for (int j = lane; j < a.k; j += 32)
          if (L.idx[j] >= 0) high = fmaxf(high, L.x[j]);
        ref_row = fmaxf(warp_max(high), ref);
      }
      double sum = 0.0;                           // loss: sum q (log q - z_j), z from ref_row; sum of exp(z_j)
      for (int j = lane; j < a.k; j += 32) {
        if (L.idx[j] < 0) continue;
        const double z = ((double)L.x[j] - (double)ref_row) * (double)a.it;
        const double lq = OP == kRenorm ? ((double)L.v[j] - sh.list_max) * (double)a.it : (double)L.v[j];
        const double q = L.q[j];
        if (!(q == 0.0)) loss += q * (lq - z);
        if (OP == kTail) {
          bool count = true;
          if (sh.repeats)
            for (int i = 0; i < j; ++i) count = count && L.idx[i] != L.idx[j];
          if (count) sum += exp(z);
        }
      }
      loss = warp_sum(loss);
      if (OP == kTail) {
        sum = warp_sum(sum);
        S_row = sum + (Sd != 0.0 ? Sd * (ref == ref_row ? 1.0 : exp(((double)ref - (double)ref_row) * (double)a.it)) : 0.0);
        if (Sd == 0.0) rho = 0.0;                 // no entry is left for the rest
      }
    }
    double log_s = 0.0;
    if constexpr (GRAD) {
      const double itd = (double)a.it;
      double ent = 0.0;
      if (w_h != 0.0f) {
        log_s = log(S_row);
        ent = (double)(float)(log(S_raw) - 0.6931471805599453 * (Td / S_raw));
      }
      const double A_list = OP == kLogprob ? -itd * ((double)w + (double)w_h * ent)
                            : itd * (double)w * (OP == kRenorm ? Q : Q + rho);
      // the gradient at the list's entries, in 64 bits: in the place of their logits
      const double inv = 1.0 / S_row;
      auto entry = [&](float x, double add) {
        const double z = ((double)x - (double)ref_row) * itd, p = exp(z) * inv;
        double g = p * A_list + itd * add;
        if (OP == kLogprob && w_h != 0.0f && p != 0.0) g -= itd * (double)w_h * p * (z - log_s);
        return (float)g;
      };
      if constexpr (LIST) {
        const double per = OP == kRenorm ? -(double)w / sh.list_sum : -(double)w;
        for (int j = lane; j < a.k; j += 32) {
          const int e = L.idx[j];
          if (e < 0 || !row.owns(e)) continue;
          double add = 0.0;
          if (Q != 0.0) {
            if (!sh.repeats) add = per * L.q[j];
            else
              for (int i = 0; i < a.k; ++i)
                if (L.idx[i] == e) add += per * L.q[i];
          }
          L.v[j] = entry(L.x[j], add);
        }
      } else if (lane == 0 && sh.target >= 0) {
        sh.g_target = entry(sh.x_target, (double)w);
      }
      if (!near) {                                // the factors, where the short way above has none
        double A, Bl = 0.0;
        if (OP == kLogprob) {
          A = A_list;
          Bl = -itd * (double)w_h * 0.6931471805599453;
        } else if (OP == kRenorm) {
          A = A_list;
        } else {
          const double Rr = Sd == 0.0 ? 0.0 : Sd / S_row * (ref == ref_row ? 1.0 : exp(((double)ref - (double)ref_row) * itd));
          A = itd * (double)w * ((Q + rho) * Rr - rho);
        }
        if (lane == 0) {
          dense_factors(sh, ref, Sd, A, Bl, a);
          sh.none = S_row == 0.0 || (w == 0.0f && w_h == 0.0f) || (LIST && sh.empty);
        }
        arrive(&sh.factors);
      }
      arrive(&sh.ready);
    }
    if (lane == 0 && part == 0) {
      log_s = log(S_row);
      if constexpr (OP == kLogprob) {
        if (a.out)
          a.out[r] = sh.target < 0     ? 0.0f
                     : S_row == 0.0 ? -INFINITY
                                    : (float)(((double)sh.x_target - (double)ref) * (double)a.it - log_s);
        if (a.entropy) a.entropy[r] = S_row == 0.0 ? 0.0f : (float)(log(S_raw) - 0.6931471805599453 * (Td / S_raw));
      } else if constexpr (OP == kRenorm) {
        a.out[r] = Q == 0.0 ? 0.0f
                            : (float)(loss / sh.list_sum - log(sh.list_sum) + (S_row == 0.0 ? (double)INFINITY : log_s));
      } else {
        if (sh.empty || (Q == 0.0 && rho == 0.0)) loss = 0.0;
        else if (S_row == 0.0) loss = Q != 0.0 ? (double)INFINITY : 0.0;
        else {
          loss += (Q + rho) * log_s;
          if (!(rho == 0.0)) loss += rho * (log(rho) - ((double)ref - (double)ref_row) * (double)a.it - log(Sd));
        }
        a.out[r] = (float)loss;
      }
      if (a.stats) {
        float* st = a.stats + (int64_t)r * (OP == kTail ? 4 : 2);
        st[0] = ref_row;
        st[1] = (float)S_row;
        if (OP == kTail) {
          st[2] = ref;
          st[3] = (float)Sd;
        }
      }

    }
    if constexpr (TOP) {
      if (lane == 0) {
        sh.nan = !(Sd == Sd);
        sh.top_ref = ref;
        sh.top_log_s = log(Sd);
      }
      wait(&sh.pushed);
    } else {
      leave();
      return;
    }
  } else {

  // Entries of the list in elements [e0, e0 + n) of the row: f(place in that range, entry).
  auto listed_in = [&](int e0, int n, auto f) {
    for (int j = lane; j < a.k; j += 32) {
      const int e = L.idx[j] - e0;
      if (L.idx[j] >= 0 && e >= 0 && e < n) f(e, j);
    }
  };
  auto hits = [&](int o) -> bool { return (sh.hit[(o / kChunk >> 5) & (kHitWords - 1)] >> ((o / kChunk) & 31)) & 1u; };

  // -- sums --------------------------------------------------------------------------------------------
  if (OP == kTail) wait(&sh.listed);
  Sums run;
  run.s = run.t = pair(0.0f, 0.0f);
  run.kind = kNone;
  run.ref = 0.0f;
  run.gaps = false;
  typename Elem<T>::Max high[U];
  if (TOP) {
#pragma unroll
    for (int u = 0; u < U; ++u) high[u] = Elem<T>::least();
  }
  for (int left = own - warp * kChunk; left > 0; left -= step) {
    const int o = own - left;                     // first vector of the chunk
    const bool hit = OP == kTail && hits(o);
    uint4* chunk = RES ? buf + o : buf;
    uint4 v[U];
    if constexpr (RES) {
      copy_wait<kAhead - 1>();
      request(left - kAhead * step);
      if (!hit) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = chunk[u * 32 + lane];
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = nx[u];
      request(left - step);
      if (hit) {
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (left >= kChunk || u * 32 + lane < left) chunk[u * 32 + lane] = v[u];
      }
    }
    if (hit) {                                    // the list's entries leave the sums
      T* el = reinterpret_cast<T*>(chunk);
      __syncwarp();
      listed_in(row.head + (row.v0 + o) * N, min(kChunk, left) * N, [&](int e, int) { el[e] = Elem<T>::from(-INFINITY); });
      __syncwarp();
    }
    if (TOP) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (left >= kChunk || u * 32 + lane < left) Elem<T>::rise(high[u], v[u]);
    }
    if (hit) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = chunk[u * 32 + lane];
    }
    if (left < kChunk) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * 32 + lane >= left) v[u] = Elem<T>::nothing();
    }
    sums_add<T, U>(run, v, a, hit || left < kChunk);
  }
  if (warp == 0 && __any_sync(kFull, edge >= 0)) {   // the entries before the first and after the last vector
    float x[N];
    x[0] = x_edge;
    if (OP == kTail && edge >= 0)
      for (int j = 0; j < a.k; ++j)
        if (L.idx[j] == edge) x[0] = -INFINITY;
#pragma unroll
    for (int i = 1; i < N; ++i) x[i] = -INFINITY;
    uint4 v[U];
    v[0] = Elem<T>::pack(x);
#pragma unroll
    for (int u = 1; u < U; ++u) v[u] = Elem<T>::nothing();
    sums_add<T, U>(run, v, a, true);
  }
  {                                               // the lanes' sums together, to the CTAs of the row
    float s0, s1, t0, t1;
    unpair(run.s, &s0, &s1);
    unpair(run.t, &t0, &t1);
    s0 = warp_sum(s0 + s1);
    t0 = warp_sum(t0 + t1);
    if (run.kind == kNan) {
      run.kind = kNear;
      run.ref = 0.0f;
      s0 = t0 = NAN;
    }
    started();
    // The gradient may take the logits' place, so that no CTA of the row begins it before the others have read
    // what they need of it.
    if (GRAD && C > 1) wait(&sh.gathered);
    const float4 sums = make_float4(run.ref, s0, t0, __int_as_float(run.kind));
    if (C == 1) {                                 // (no asynchronous store outside a cluster launch: it is illegal there)
      if (lane == 0) sh.part[warp] = sums;
      arrive(&sh.sums);
    } else if (lane < (GRAD ? C : 1)) {
      peer_send(&sh.part[part * W + warp], &sh.sums, lane, sums);
    }
  }

  // -- candidates for the alternatives ------------------------------------------------------------------
  // The largest entry of a part is an entry, so a value that k parts reach is a lower bound of the
  // slice's, and so of the row's, k-th largest. The warps look for the largest such value by bisection on
  // the keys (a value that a few more parts reach will do), and the CTAs take the largest of theirs. Then
  // the parts that reach it are read again, from L2, shared out among the warps: the likely tokens of a
  // vocabulary sorted by frequency all lie in one warp's chunks.
  if constexpr (TOP) {
    auto meet = [&]() { asm volatile("bar.sync 1, %0;" ::"r"(W * 32) : "memory"); };
    uint32_t key[U], mx = 0, mn = 0xffffffffu, valid = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      key[u] = order_key(Elem<T>::top(high[u]));
      mx = max(mx, key[u]);
      if (key[u] > kKeyNegInf) {
        mn = min(mn, key[u]);
        ++valid;
      }
    }
    mx = __reduce_max_sync(kFull, mx);
    mn = __reduce_min_sync(kFull, mn);
    valid = __reduce_add_sync(kFull, valid);
    if (warp == 0 && lane < 8) sh.reach[0][lane] = 0;   // (of warps that are not there, too)
    if (lane == 0) {
      sh.tops[warp] = mx;
      sh.least[warp] = mn;
      sh.reach[1][warp] = valid;
    }
    if (warp == 0 && lane >= W && lane < 8) sh.reach[1][lane] = 0;
    meet();
    valid = 0;
    for (int q = 0; q < W; ++q) {
      mx = max(mx, sh.tops[q]);
      mn = min(mn, sh.least[q]);
      valid += sh.reach[1][q];
    }
    uint32_t bound = kKeyNegInf + 1;
    if ((int)valid >= a.k) {
      // two bits of it a round: one reduction per warp and one barrier
      const int bits = (33 - __clz(mx ^ mn)) & ~1;    // below these, rounded up to pairs, the keys agree
      uint32_t res = bits == 32 ? 0u : mx >> bits << bits;
      int turn = 0;
      for (int b = bits - 2; b >= 0; b -= 2) {
        uint32_t n = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (uint32_t i = 1; i < 4; ++i) n += (key[u] > kKeyNegInf && key[u] >= res + (i << b)) << (10 * (i - 1));
        n = __reduce_add_sync(kFull, n);
        if (lane == 0) sh.reach[turn][warp] = n;
        meet();
        const uint4 lo = *reinterpret_cast<const uint4*>(&sh.reach[turn][0]), hi = *reinterpret_cast<const uint4*>(&sh.reach[turn][4]);
        n = lo.x + lo.y + lo.z + lo.w + hi.x + hi.y + hi.z + hi.w;
        turn ^= 1;
        const int n1 = n & 1023, n2 = (n >> 10) & 1023, n3 = (int)(n >> 20);
        const int up = n3 >= a.k ? 3 : n2 >= a.k ? 2 : n1 >= a.k ? 1 : 0;
        const int got = up == 3 ? n3 : up == 2 ? n2 : n1;
        res += (uint32_t)up << b;
        if (up && got <= a.k + a.k / 4 + 2) break;
      }
      bound = max(bound, res);
    }
    if (C > 1) {
      if (warp == 0 && lane < C) {
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer(&sh.bounds[part], lane)), "r"(bound) : "memory");
        peer_arrive(&sh.bounded, lane);
      }
      wait(&sh.bounded);
      for (int q = 0; q < C; ++q) bound = max(bound, sh.bounds[q]);
    }
    if (lane == 0 && warp == 0) sh.bounds[0] = bound;   // (what others may still read there does not change theirs)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t who = __ballot_sync(kFull, key[u] >= bound);
      int first = 0;
      if (lane == 0 && who) first = atomicAdd(&sh.owners, __popc(who));
      first = __shfl_sync(kFull, first, 0);
      if (key[u] >= bound) owners[first + __popc(who & lanemask_lt())] = (uint16_t)(warp << 7 | u << 5 | lane);
    }
    meet();
    const int n_own = sh.owners, chunks = (own + kChunk - 1) / kChunk;
    const int most = (chunks + W - 1) / W;        // vectors of a part
    const int width = most <= 4 ? 4 : most <= 8 ? 8 : most <= 16 ? 16 : 32;
    for (int q = (warp * 32 + lane) / width; q < n_own; q += W * 32 / width) {
      const int o = owners[q], at_w = o >> 7, at_u = (o >> 5) & 3, at_l = o & 31;
      for (int j = lane % width; j < most; j += width) {
        const int i = (at_w + W * j) * kChunk + at_u * 32 + at_l;
        if (i >= own) break;
        float x[N];
        Elem<T>::unpack(ld_row(row.vec() + row.v0 + i), x);
        uint32_t hits = 0;
#pragma unroll
        for (int b = 0; b < N; ++b) hits |= (order_key(x[b]) >= bound ? 1u : 0u) << b;
        if (hits == 0) continue;
        uint32_t n = peer_places(&top, __popc(hits), C == 1);
#pragma unroll
        for (int b = 0; b < N; ++b)
          if ((hits >> b) & 1u) peer_put(&top, n++, order_key(x[b]), row.head + (row.v0 + i) * N + b, C == 1);
      }
    }
    if (edge >= 0 && order_key(x_edge) >= bound) peer_put(&top, peer_places(&top, 1, C == 1), order_key(x_edge), edge, C == 1);
    if (C > 1) {
      asm volatile("fence.acq_rel.cluster;" ::: "memory");
      __syncwarp();
      if (lane == 0) peer_arrive(&sh.pushed, 0);
    } else {
      arrive(&sh.pushed);
    }
    if (part != 0) {
      leave();
      return;
    }
    wait(&sh.pushed);
  }

  // -- gradient ------------------------------------------------------------------------------------------
  if constexpr (GRAD) {
    at = row.vec() + row.v0 + warp * kChunk + lane;
    if (!RES) request(own - warp * kChunk);
    wait(&sh.factors);
    const float kf = sh.k, A = sh.A, Bl = sh.Bl, ref = sh.ref;
    const bool away = sh.away, none = sh.none;
    T* dx = static_cast<T*>(a.dlogits) + (int64_t)r * a.dstride;
    const bool in_step = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(row.x)) & 15u) == 0;
    const bool plain = in_step && !away && !none;
    uint4* dvec = reinterpret_cast<uint4*>(dx + row.head) + row.v0;
    const f2 c2 = pair(a.c, a.c), nk = pair(-kf, -kf), A2 = pair(A, A), B2 = pair(Bl, Bl);
    auto grad = [&](uint4 v, auto far) {             // far: the difference first
      float x[N];
      Elem<T>::unpack(v, x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float q0, q1;
        f2 q, g = A2;
        if constexpr (far.value) {
          q0 = max_nan((x[i] - ref) * a.c, -kFarBits) - kf;
          q1 = max_nan((x[i + 1] - ref) * a.c, -kFarBits) - kf;
        } else {
          q = fma2(pair(x[i], x[i + 1]), c2, nk);
          unpair(q, &q0, &q1);
        }
        if (OP == kLogprob && Bl != 0.0f) g = fma2(pair(max_nan(q0, -kFarBits), max_nan(q1, -kFarBits)), B2, A2);
        unpair(mul2(pair(ex2(q0), ex2(q1)), g), &x[i], &x[i + 1]);
      }
      return Elem<T>::pack(x);
    };
    auto grad_one = [&](float x) {
      const float q = away ? max_nan((x - ref) * a.c, -kFarBits) - kf : fmaf(x, a.c, -kf);
      return Elem<T>::from(ex2(q) * (Bl != 0.0f ? fmaf(max_nan(q, -kFarBits), Bl, A) : A));
    };
    // The whole chunks without entries of the list, in a loop of their own that holds little else (one loop
    // for all chunks took 160 instructions per chunk more); the others after it.
    uint32_t rest = 0xffffffffu;
    if constexpr (RES) {
      if (plain) {
        const int target_chunk = LIST ? -1 : sh.target < row.head ? -1 : ((sh.target - row.head) / N - row.v0) >> kChunkLog;
        const uint4* from = buf + warp * kChunk + lane;
        uint4* to = dvec + warp * kChunk + lane;
        rest = 0;
        int c = warp;
        for (int left = own - warp * kChunk; left > 0; left -= step, c += W, from += step, to += step) {
          bool apart = left < kChunk;
          if (LIST) apart |= (sh.hit[(c >> 5) & (kHitWords - 1)] >> (c & 31)) & 1u;
          else apart |= c == target_chunk;
          if (apart) {
            rest |= 1u << (c / W);
            continue;
          }
          uint4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) v[u] = from[u * 32];
#pragma unroll
          for (int u = 0; u < U; ++u) __stcs(to + u * 32, grad(v[u], std::false_type{}));
        }
      }
    }
    for (int left = own - warp * kChunk; left > 0; left -= step, rest >>= RES ? 1 : 0) {
      if (RES && !(rest & 1u)) continue;
      const int o = own - left, e0 = row.head + (row.v0 + o) * N;   // first vector and element
      uint4* chunk = RES ? buf + o : buf;
      T* el = reinterpret_cast<T*>(chunk);
      uint4 v[U];
      if constexpr (!RES) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = nx[u];
        request(left - step);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = chunk[u * 32 + lane];
      }
      uint4* to = dvec + o + lane;
      bool hit;
      if (LIST) hit = hits(o);
      else hit = sh.target >= e0 && sh.target < e0 + kChunk * N;
      if (away) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = grad(v[u], std::true_type{});
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = grad(v[u], std::false_type{});
      }
      if (plain && !hit) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u * 32 + lane < left) __stcs(to + u * 32, v[u]);
      } else {
        // through shared memory: the list's entries over the dense gradient
        const int n = min(left, kChunk);
        if (!RES) __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u * 32 + lane < n) chunk[u * 32 + lane] = none ? make_uint4(0, 0, 0, 0) : v[u];
        __syncwarp();
        if (!none) {
          if constexpr (LIST) {
            if (hit) {
              wait(&sh.ready);
              listed_in(e0, n * N, [&](int e, int j) { el[e] = Elem<T>::from(L.v[j]); });
            }
          } else {
            if (hit) {
              wait(&sh.ready);
              if (lane == 0 && sh.target - e0 < n * N) el[sh.target - e0] = Elem<T>::from(sh.g_target);
            }
          }
          __syncwarp();
        }
        if (in_step) {
          for (int u = lane; u < n; u += 32) __stcs(to + u - lane, chunk[u]);
        } else {
          for (int e = lane; e < n * N; e += 32) dx[e0 + e] = el[e];
        }
      }
    }
    if (edge >= 0) {
      T g = none ? Elem<T>::from(0.0f) : grad_one(x_edge);
      if (!none) {
        wait(&sh.ready);
        if constexpr (LIST) {
          for (int j = 0; j < a.k; ++j)
            if (L.idx[j] == edge) g = Elem<T>::from(L.v[j]);
        } else {
          if (sh.target == edge) g = Elem<T>::from(sh.g_target);
        }
      }
      dx[edge] = g;
    }
  }
  if constexpr (!TOP) {
    leave();
    return;
  }
  }

  // -- the alternatives, by all warps of the first CTA ---------------------------------------------------
  if constexpr (TOP) {
    const int tid = threadIdx.x, B = blockDim.x;
    __syncthreads();
    if (top.count > kCand || sh.nan) {
      const Row<T> whole(row.x, a.vocab, 0, 1, 0u);
      exact_top(whole, a.k, sh.bounds[0], top, sh.scratch);
    }
    int n = top.count;
    unsigned long long* cand = top.cand;
    if (n > 192 && n > 2 * a.k) {
      // too many to rank one against all: those from their own k-th key on, or a little below
      uint32_t res = 0;
      int reached = n;
      for (int b = 31; b >= 0; --b) {
        const uint32_t trial = res | (1u << b);
        int c = 0;
        for (int i = tid; i < n; i += B) c += (uint32_t)(cand[i] >> 32) >= trial;
        c = block_count(c, sh.scratch);
        if (c >= a.k) {
          res = trial;
          reached = c;
          if (c <= a.k + a.k / 2 + 16) break;
        }
      }
      unsigned long long* to = reinterpret_cast<unsigned long long*>(dyn);
      if (reached <= W * kChunk * 2) {
        __syncthreads();
        if (tid == 0) sh.scratch[0] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += B)
          if ((uint32_t)(cand[i] >> 32) >= res) to[atomicAdd(&sh.scratch[0], 1)] = cand[i];
        __syncthreads();
        cand = to;
        n = reached;
      }
    }
    // rank of a candidate = how many are larger; `per` neighbouring lanes share one
    int per = 1;
    while (per < 32 && 2 * per * n <= B) per *= 2;
    for (int base = 0; base < n; base += B / per) {
      const int i = base + tid / per;
      int above = 0;
      const unsigned long long me = i < n ? cand[i] : 0ull;
      for (int j = tid % per; j < n; j += per) above += cand[j] > me;
      for (int d = per >> 1; d > 0; d >>= 1) above += __shfl_xor_sync(kFull, above, d);
      if (i < n && tid % per == 0 && above < a.k) {
        const int e = (int)~(uint32_t)me;
        const int64_t o = (int64_t)r * a.k + above;
        a.top_idx[o] = e;
        a.top_val[o] = (float)(((double)Elem<T>::to(row.x[e]) - (double)sh.top_ref) * (double)a.it - sh.top_log_s);
      }
    }
    for (int j = n + tid; j < a.k; j += B) {
      a.top_idx[(int64_t)r * a.k + j] = -1;
      a.top_val[(int64_t)r * a.k + j] = -INFINITY;
    }
    leave();
  }
}

// ---- launch -----------------------------------------------------------------------------------------

constexpr size_t kPlainBytes = 32 << 10;          // dynamic shared memory that needs no leave beside the static part
constexpr int64_t kSliceBytes = 64 << 10;         // three or four CTAs per SM
constexpr int64_t kSliceMost = 200 << 10;         // one CTA per SM

// The leave for a launch of `smem` bytes. It belongs to the kernel, not to the call: every call sets the most that any
// call of the kernel needs, so that one thread's small call does not take back what another's launch is about to use.
template <class K>
bool voc_leave(K* kernel, size_t smem, size_t most) {
  if (smem <= kPlainBytes) return true;
  if (smem <= most && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

template <class T, int OP, int MODE, bool RES, bool TOP>
int voc_stream_launch(VocArgs a, int64_t nv, int split, cudaStream_t st) {
  const int64_t own = cdiv(nv, split), chunks = cdiv(own, kChunk);
  int warps = (int)(chunks < kRowWarps ? (chunks > 0 ? chunks : 1) : kRowWarps);
  a.split = split;
  a.slice = (int32_t)(chunks * kChunk);
  a.inv_split = (uint32_t)(((1ull << 32) + split - 1) / split);
  auto bytes = [](size_t vectors, int w, int k) {
    return vectors * 16 + (OP == kLogprob ? 0 : List::bytes(k)) + (TOP ? (size_t)w * 256 + sizeof(TopShared) : 0);
  };
  const size_t smem = bytes(RES ? a.slice : warps * kChunk, warps, a.k);
  const size_t most = bytes(RES ? kSliceMost / 16 + kChunk : kRowWarps * kChunk, kRowWarps, GSPARSE_MAX_ALTERNATIVES);
  auto* kernel = voc_stream_kernel<T, OP, MODE, RES, TOP>;
  if (!voc_leave(kernel, smem, most)) return GSPARSE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * split));
  cfg.blockDim = dim3((unsigned)((warps + 1) * 32));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return GSPARSE_ERR_CUDA;
  }
  return launch_status();
}

template <class T, int OP, int MODE, bool TOP>
int voc_stream(const VocArgs& a, cudaStream_t st) {
  const int64_t nv = cdiv(a.vocab, Elem<T>::N);
  // few rows: split each over up to 8 CTAs, as long as a CTA keeps 256 vectors
  int split = 1;
  while (split < 8 && (int64_t)a.rows * split < 2 * sm_count() && nv / (2 * split) >= 256) split *= 2;
  if constexpr (MODE == kFused) {
    // Powers of two: clusters of 3 and 6 find their places later than those of 2 and 4 (2048 x 50021 fp16: 212
    // us in three slices of 33 KB, 152 in two of 50; 8192 x 128000 bf16: 1022 us in six, 888 in four).
    while (split < 8 && nv * 16 > split * kSliceBytes) split *= 2;
    if (nv * 16 <= split * kSliceMost) return voc_stream_launch<T, OP, MODE, true, false>(a, nv, split, st);
  }
  return voc_stream_launch<T, OP, MODE, false, TOP>(a, nv, split, st);
}

template <class T, int OP>
int voc_backward(VocArgs a, cudaStream_t st) {
  const int64_t nv = cdiv(a.vocab, Elem<T>::N);
  // few rows: split each over up to 8 CTAs, as long as a CTA keeps 512 vectors
  int split = 1;
  while (split < 8 && (int64_t)a.rows * split < 2 * sm_count() && nv / (2 * split) >= 512) split *= 2;
  a.split = split;
  a.inv_split = (uint32_t)(((1ull << 32) + split - 1) / split);
  int threads = 64;
  while (threads < kVocThreads && (int64_t)threads * kUnroll * split < nv) threads *= 2;
  const size_t smem = ring_bytes(threads) + List::bytes(OP == kLogprob ? a.k + 1 : a.k);
  auto* kernel = voc_backward_kernel<T, OP>;
  if (!voc_leave(kernel, smem, ring_bytes(kVocThreads) + List::bytes(GSPARSE_MAX_ALTERNATIVES + 1))) return GSPARSE_ERR_CUDA;
  launch(kernel, (unsigned)((int64_t)a.rows * split), (unsigned)threads, smem, st, a);
  return launch_status();
}

template <class T, int OP, int MODE, bool TOP>
int voc_of_type(const VocArgs& a, cudaStream_t st) {
  if constexpr (MODE == kBackward) return voc_backward<T, OP>(a, st);
  else return voc_stream<T, OP, MODE, TOP>(a, st);
}

template <int OP, int MODE, bool TOP = false>
int voc_by_type(int32_t dtype, const VocArgs& a, cudaStream_t st) {
  if (dtype == GSPARSE_F32) return voc_of_type<float, OP, MODE, TOP>(a, st);
  if (dtype == GSPARSE_BF16) return voc_of_type<__nv_bfloat16, OP, MODE, TOP>(a, st);
  return voc_of_type<__half, OP, MODE, TOP>(a, st);
}

bool voc_dtype(int32_t t) { return t == GSPARSE_F32 || t == GSPARSE_BF16 || t == GSPARSE_F16; }

// Arguments common to the four calls.
int voc_common(VocArgs& a, const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t stride,
               float inv_temperature, void* dlogits, int64_t dstride, int32_t* d_status) {
  if (!voc_dtype(dtype) || rows < 0 || vocab < 1 || stride < 0) return GSPARSE_ERR_INVALID_ARG;
  if (!(inv_temperature > 0.0f) || !isfinite(inv_temperature)) return GSPARSE_ERR_INVALID_ARG;
  if (inv_temperature < 0x1p-64f || inv_temperature > 0x1p64f) return GSPARSE_ERR_UNSUPPORTED;
  if (rows >= (1 << 26) || vocab > GSPARSE_MAX_VOCAB) return GSPARSE_ERR_UNSUPPORTED;
  const uintptr_t align = dtype == GSPARSE_F32 ? 3 : 1;
  if (rows > 0 && !logits) return GSPARSE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & align) || (reinterpret_cast<uintptr_t>(dlogits) & align))
    return GSPARSE_ERR_INVALID_ARG;
  if (dlogits && rows > 1 && dstride < vocab) return GSPARSE_ERR_INVALID_ARG;
  if (dlogits == logits && dlogits && rows > 1 && dstride != stride) return GSPARSE_ERR_INVALID_ARG;
  const double c = (double)inv_temperature * 1.4426950408889634;
  a.c = (float)c;
  a.c_lo = (float)(c - (double)a.c);
  a.fine = (float)((double)a.c_lo / (double)a.c * 0.6931471805599453);
  a.inv_c = 1.0 / (double)a.c;
  a.it = inv_temperature;
  a.logits = logits;
  a.dlogits = dlogits;
  a.stride = stride;
  a.dstride = dstride;
  a.rows = (int32_t)rows;
  a.vocab = (int32_t)vocab;
  a.d_status = d_status;
  return GSPARSE_OK;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" {

int gsparse_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                           float inv_temperature, const int32_t* targets, float* logprob, float* entropy,
                           float* stats, int32_t top_k, int32_t* top_idx, float* top_logprob, void* dlogits,
                           int64_t dlogits_stride, const float* grad_logprob, const float* grad_entropy,
                           int32_t* d_status, gsparse_stream stream) {
  VocArgs a{};
  const int st = voc_common(a, logits, dtype, rows, vocab, row_stride, inv_temperature, dlogits, dlogits_stride, d_status);
  if (st != GSPARSE_OK) return st;
  if (top_k < 0 || top_k > vocab || (top_k > 0 && rows > 0 && (!top_idx || !top_logprob))) return GSPARSE_ERR_INVALID_ARG;
  if (top_k > GSPARSE_MAX_ALTERNATIVES) return GSPARSE_ERR_UNSUPPORTED;
  if (rows > 0 && logprob && !targets) return GSPARSE_ERR_INVALID_ARG;
  if (!dlogits && (grad_logprob || grad_entropy)) return GSPARSE_ERR_INVALID_ARG;
  if (grad_logprob && !targets) return GSPARSE_ERR_INVALID_ARG;
  if (rows == 0) return GSPARSE_OK;
  a.targets = targets;
  a.out = logprob;
  a.entropy = entropy;
  a.stats = stats;
  a.k = top_k;
  a.top_idx = top_idx;
  a.top_val = top_logprob;
  a.weight = grad_logprob;
  a.weight_entropy = grad_entropy;
  cudaStream_t s = (cudaStream_t)stream;
  if (top_k && dlogits) {                         // the alternatives first: the gradient may take the logits' place
    VocArgs t = a;
    t.out = t.entropy = t.stats = nullptr;
    const int e = voc_by_type<kLogprob, kForward, true>(dtype, t, s);
    if (e != GSPARSE_OK) return e;
  }
  if (dlogits) return voc_by_type<kLogprob, kFused>(dtype, a, s);
  return top_k ? voc_by_type<kLogprob, kForward, true>(dtype, a, s) : voc_by_type<kLogprob, kForward>(dtype, a, s);
}

int gsparse_token_logprobs_backward(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                                    int64_t row_stride, float inv_temperature, const float* stats,
                                    const int32_t* targets, const float* grad_logprob, const float* entropy,
                                    const float* grad_entropy, int32_t top_k, const int32_t* top_idx,
                                    const float* grad_top, void* dlogits, int64_t dlogits_stride,
                                    int32_t* d_status, gsparse_stream stream) {
  VocArgs a{};
  const int st = voc_common(a, logits, dtype, rows, vocab, row_stride, inv_temperature, dlogits, dlogits_stride, d_status);
  if (st != GSPARSE_OK) return st;
  if (top_k < 0 || top_k > vocab || (top_k > 0 && rows > 0 && (!top_idx || !grad_top))) return GSPARSE_ERR_INVALID_ARG;
  if (top_k > GSPARSE_MAX_ALTERNATIVES) return GSPARSE_ERR_UNSUPPORTED;
  if (rows > 0 && (!stats || !dlogits)) return GSPARSE_ERR_INVALID_ARG;
  if ((grad_logprob && !targets) || (grad_entropy && !entropy)) return GSPARSE_ERR_INVALID_ARG;
  if (rows == 0) return GSPARSE_OK;
  a.targets = targets;
  a.stats_in = stats;
  a.entropy_in = entropy;
  a.weight = grad_logprob;
  a.weight_entropy = grad_entropy;
  a.k = top_k;
  a.list_idx = top_idx;
  a.list_val = grad_top;
  return voc_by_type<kLogprob, kBackward>(dtype, a, (cudaStream_t)stream);
}

int gsparse_distill_topk(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                         float inv_temperature, const int32_t* teacher_idx, const void* teacher_val,
                         int32_t val_dtype, int32_t k, int32_t mode, float* loss, float* stats, void* dlogits,
                         int64_t dlogits_stride, const float* grad_loss, int32_t* d_status,
                         gsparse_stream stream) {
  VocArgs a{};
  const int st = voc_common(a, logits, dtype, rows, vocab, row_stride, inv_temperature, dlogits, dlogits_stride, d_status);
  if (st != GSPARSE_OK) return st;
  if (!voc_dtype(val_dtype) || k < 1 || (mode != GSPARSE_DISTILL_RENORM && mode != GSPARSE_DISTILL_TAIL))
    return GSPARSE_ERR_INVALID_ARG;
  if (k > GSPARSE_MAX_ALTERNATIVES) return GSPARSE_ERR_UNSUPPORTED;
  if (rows > 0 && (!teacher_idx || !teacher_val || !loss)) return GSPARSE_ERR_INVALID_ARG;
  if (rows > 0 && ((dlogits != nullptr) != (grad_loss != nullptr))) return GSPARSE_ERR_INVALID_ARG;
  if (rows == 0) return GSPARSE_OK;
  a.list_idx = teacher_idx;
  a.list_val = teacher_val;
  a.val_dtype = val_dtype;
  a.k = k;
  a.out = loss;
  a.stats = stats;
  a.weight = grad_loss;
  cudaStream_t s = (cudaStream_t)stream;
  if (mode == GSPARSE_DISTILL_TAIL)
    return dlogits ? voc_by_type<kTail, kFused>(dtype, a, s) : voc_by_type<kTail, kForward>(dtype, a, s);
  return dlogits ? voc_by_type<kRenorm, kFused>(dtype, a, s) : voc_by_type<kRenorm, kForward>(dtype, a, s);
}

int gsparse_distill_topk_backward(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                                  int64_t row_stride, float inv_temperature, const float* stats,
                                  const int32_t* teacher_idx, const void* teacher_val, int32_t val_dtype,
                                  int32_t k, int32_t mode, const float* grad_loss, void* dlogits,
                                  int64_t dlogits_stride, int32_t* d_status, gsparse_stream stream) {
  VocArgs a{};
  const int st = voc_common(a, logits, dtype, rows, vocab, row_stride, inv_temperature, dlogits, dlogits_stride, d_status);
  if (st != GSPARSE_OK) return st;
  if (!voc_dtype(val_dtype) || k < 1 || (mode != GSPARSE_DISTILL_RENORM && mode != GSPARSE_DISTILL_TAIL))
    return GSPARSE_ERR_INVALID_ARG;
  if (k > GSPARSE_MAX_ALTERNATIVES) return GSPARSE_ERR_UNSUPPORTED;
  if (rows > 0 && (!teacher_idx || !teacher_val || !stats || !dlogits || !grad_loss)) return GSPARSE_ERR_INVALID_ARG;
  if (rows == 0) return GSPARSE_OK;
  a.list_idx = teacher_idx;
  a.list_val = teacher_val;
  a.val_dtype = val_dtype;
  a.k = k;
  a.stats_in = stats;
  a.weight = grad_loss;
  if (mode == GSPARSE_DISTILL_TAIL) return voc_by_type<kTail, kBackward>(dtype, a, (cudaStream_t)stream);
  return voc_by_type<kRenorm, kBackward>(dtype, a, (cudaStream_t)stream);
}

}  // extern "C"

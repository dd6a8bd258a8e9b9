// Losses over vocabulary rows: log probabilities of given tokens with the row's entropy and its most
// likely tokens, and distillation from a teacher's (index, value) list, each with the gradient of the
// logits in the same call or as a pass of its own.
//
// With z = x * it (it = 1 / temperature), M = max x, c = it * log2(e):
//   S = sum 2^((x - M) c),  T = sum 2^((x - M) c) (x - M) c,  p = 2^((x - M) c - log2 S),
//   entropy = ln2 (log2 S - T / S),  log p_t = (x_t - M) it - ln S,
// so one pass over a row with a running maximum gives everything but the gradient, and the gradient
// of either loss is p (A + B log2 p) per entry plus a few entries of the row's list, which are
// computed and written apart after the dense pass.
//
// One thread-block cluster of C CTAs takes a row, each CTA a slice of it; the CTAs exchange their
// (M, S, T) through distributed shared memory. C = 1 when there are rows enough to fill the GPU.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"

namespace gs {
namespace {

namespace cg = cooperative_groups;

constexpr int kVocThreads = 512;
constexpr int kVocWarps = kVocThreads / 32;
constexpr int kVocUnroll = 4;                     // 16-byte loads in flight per thread
constexpr int kCand = 1024;                       // candidates for the alternatives, per CTA and in all
constexpr int kList = GSPARSE_MAX_ALTERNATIVES + 1;   // a row's list and its target
constexpr int kTable = 1024;                      // hash table over the list (load <= 1/4)
constexpr int kFilterWords = 512;                 // one bit per vector of the row, modulo 16384

constexpr float kLowest = -3.402823466e38f;       // the maximum of a row that holds nothing but -inf
constexpr float kFarBits = 1.0e4f;                // 2^-10^4 = 0: exponents are clamped here, so that
                                                  // 0 * exponent stays 0 where the logit is -inf

enum { kLogprob = 0, kRenorm = 1, kTail = 2 };    // what is computed
enum { kForward = 0, kFused = 1, kBackward = 2 }; // loss; loss and gradient; gradient from saved statistics

struct VocArgs {
  const void* logits;
  void* dlogits;
  int64_t stride, dstride;       // elements
  int32_t rows, vocab, split;    // split = CTAs per row
  int32_t k;                     // list length: alternatives wanted (forward), given (backward), or the teacher's
  int32_t val_dtype;
  float it, c, c_lo, far;        // c + c_lo = it log2(e); far = kFarBits / c
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
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
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
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
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

struct Scratch {
  float f[kVocWarps];
  double a[kVocWarps], b[kVocWarps];
  int i[kVocWarps];
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}

// Each leaves its scratch free for the next call (the sync at the start).
__device__ __forceinline__ float block_max(float v, Scratch& sh) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.f[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float m = sh.f[0];
  for (int w = 1; w < nw; ++w) m = fmaxf(m, sh.f[w]);
  return m;
}
__device__ __forceinline__ void block_sum2(double& x, double& y, Scratch& sh) {
  x = warp_sum(x);
  y = warp_sum(y);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.a[threadIdx.x >> 5] = x;
    sh.b[threadIdx.x >> 5] = y;
  }
  __syncthreads();
  const int nw = blockDim.x >> 5;
  x = sh.a[0];
  y = sh.b[0];
  for (int w = 1; w < nw; ++w) {
    x += sh.a[w];
    y += sh.b[w];
  }
}
__device__ __forceinline__ int block_count(int v, Scratch& sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.i[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  int n = 0;
  for (int w = 0; w < nw; ++w) n += sh.i[w];
  return n;
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
  __device__ __forceinline__ Row(const T* p, int vocab, int part, int split) : x(p), V(vocab) {
    constexpr int N = Elem<T>::N;
    head = (int)(((16u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
    if (head > V) head = V;
    nv = (V - head) / N;
    v0 = (int)((int64_t)nv * part / split);
    v1 = (int)((int64_t)nv * (part + 1) / split);
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
  // Vector number of element e, the head being vector 0 and the body starting at 1.
  __device__ __forceinline__ int vec_of(int e) const { return e < head ? 0 : (e - head) / Elem<T>::N + 1; }
  __device__ __forceinline__ int lane_of(int e) const { return e < head ? e : (e - head) % Elem<T>::N; }
  __device__ __forceinline__ bool owns(int e) const {
    const int v = vec_of(e);
    if (v == 0) return first;
    if (v == nv + 1) return last;
    return v - 1 >= v0 && v - 1 < v1;
  }
};

// ---- running maximum and sums -----------------------------------------------------------------

struct Running {
  float m;        // largest entry so far, -inf if none (NaN is passed over; it reaches s)
  f2 s, t;        // sums over entries of e = 2^((x - ref) c) and of e (x - ref) c, ref = max(m, lowest)
};

__device__ __forceinline__ void running_init(Running& r) {
  r.m = -INFINITY;
  r.s = r.t = pair(0.0f, 0.0f);
}

// Moves the sums to the maximum m2 >= m.
__device__ __forceinline__ void running_raise(Running& r, float m2, float c) {
  const float dd = max_nan((fmaxf(r.m, kLowest) - fmaxf(m2, kLowest)) * c, -kFarBits);
  const float f = ex2(dd);
  r.t = mul2(fma2(r.s, pair(dd, dd), r.t), pair(f, f));
  r.s = mul2(r.s, pair(f, f));
  r.m = m2;
}

// Adds n entries (n even). FINE: the product with c in two parts, so that the rounding of c does
// not shift every exponent the same way (the distillation loss is a small difference of logs).
template <int NE, bool ENT, bool FINE>
__device__ __forceinline__ void running_add(Running& r, const float* x, const VocArgs& a) {
  const float ref = fmaxf(r.m, kLowest);
  const f2 nref = pair(-ref, -ref), c2 = pair(a.c, a.c);
#pragma unroll
  for (int i = 0; i < NE; i += 2) {
    float d0, d1;
    unpair(add2(pair(x[i], x[i + 1]), nref), &d0, &d1);
    const f2 d = pair(max_nan(d0, -a.far), max_nan(d1, -a.far));
    f2 q = mul2(d, c2);
    if (FINE) q = fma2(d, pair(a.c_lo, a.c_lo), q);
    float q0, q1;
    unpair(q, &q0, &q1);
    const f2 e = pair(ex2(q0), ex2(q1));
    r.s = add2(r.s, e);
    if (ENT) r.t = fma2(e, q, r.t);
  }
}

// ---- list of a row ------------------------------------------------------------------------------

struct ListShared {
  int32_t idx[kList];      // -1: absent
  float x[kList];          // the row's entry there
  float add[kList];        // what the gradient gets there besides the dense part
  uint32_t table[kTable];  // (vector + 1) << 8 | entries of that vector in the list
  uint32_t filter[kFilterWords];
  int repeats;             // an index stands in the list twice
};

__device__ __forceinline__ uint32_t table_slot(uint32_t v) { return (v * 2654435761u) >> 22; }   // kTable = 2^10

// Enters element (vector v, place l) into the table; true if it was there.
__device__ __forceinline__ bool table_add(ListShared& L, int v, int l) {
  const uint32_t tag = (uint32_t)(v + 1) << 8, bit = 1u << l;
  uint32_t s = table_slot((uint32_t)v);
  for (int n = 0; n < kTable; ++n, s = (s + 1) & (kTable - 1)) {
    const uint32_t old = atomicCAS(&L.table[s], 0u, tag | bit);
    if (old == 0u) break;
    if ((old & ~255u) == tag) return (atomicOr(&L.table[s], bit) & bit) != 0;
  }
  atomicOr(&L.filter[((uint32_t)v >> 5) & (kFilterWords - 1)], 1u << (v & 31));
  return false;
}

// Which entries of vector v are in the list.
__device__ __forceinline__ uint32_t table_mask(const ListShared& L, int v) {
  if (!((L.filter[((uint32_t)v >> 5) & (kFilterWords - 1)] >> (v & 31)) & 1u)) return 0;
  const uint32_t tag = (uint32_t)(v + 1) << 8;
  uint32_t s = table_slot((uint32_t)v);
  for (int n = 0; n < kTable; ++n, s = (s + 1) & (kTable - 1)) {
    const uint32_t w = L.table[s];
    if (w == 0u) return 0;
    if ((w & ~255u) == tag) return w & 255u;
  }
  return 0;
}

template <class T>
__device__ __forceinline__ uint4 masked(uint4 u, uint32_t mask) {
  float x[Elem<T>::N];
  Elem<T>::unpack(u, x);
#pragma unroll
  for (int i = 0; i < Elem<T>::N; ++i)
    if ((mask >> i) & 1u) x[i] = -INFINITY;
  return Elem<T>::pack(x);
}

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

// The largest key with at least k of the block's keys at or above it; 0 if there are not k valid
// keys (a key at or below -inf's is not valid). Stops as soon as exactly k are above.
__device__ uint32_t kth_key_of_block(uint32_t key, int k) {
  const bool valid = key > kKeyNegInf;
  if (__syncthreads_count(valid) < k) return 0;
  uint32_t res = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t trial = res | (1u << b);
    const int n = __syncthreads_count(valid && key >= trial);
    if (n >= k) res = trial;
    if (n == k) break;
  }
  return res;
}

// Entries of the whole row with key >= t (the CTA reads all of it).
template <class T>
__device__ int count_ge(const Row<T>& row, uint32_t t, Scratch& sh) {
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
__device__ __noinline__ void exact_top(const Row<T>& row, int k, uint32_t lower, TopShared& top, Scratch& sh) {
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
    if ((threadIdx.x & 31) == 0) sh.i[threadIdx.x >> 5] = __popc(b);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
      if (w < (int)(threadIdx.x >> 5)) before += sh.i[w];
      all += sh.i[w];
    }
    before += __popc(b & lanemask_lt());
    if (hit && found + before < need) cand_push(top, lo, e);
    found += all;
  }
  __syncthreads();
}

// ---- the kernel -----------------------------------------------------------------------------------

struct Exchange {      // what the CTAs of a row tell each other
  float m;
  double s, t;
  uint32_t kth;
};

template <bool LIST> struct ListPart { ListShared list; };
template <> struct ListPart<false> {};
template <bool TOP> struct TopPart { TopShared top; };
template <> struct TopPart<false> {};

template <class T, int OP, bool TOP, int MODE>
__global__ void __launch_bounds__(kVocThreads, 2) voc_kernel(const __grid_constant__ VocArgs a) {
  constexpr int N = Elem<T>::N, U = kVocUnroll;
  constexpr bool LIST = OP != kLogprob || MODE == kBackward;
  constexpr bool FINE = OP != kLogprob;
  constexpr bool ENT = OP == kLogprob;
  __shared__ Scratch sh;
  __shared__ Exchange ex;
  __shared__ ListPart<LIST> lp;
  __shared__ TopPart<TOP> tp;

  const int C = a.split, part = (int)(blockIdx.x % (unsigned)C), r = (int)(blockIdx.x / (unsigned)C);
  const int tid = threadIdx.x, B = blockDim.x;
  const Row<T> row(static_cast<const T*>(a.logits) + (int64_t)r * a.stride, a.vocab, part, C);
  const uint4* vec = row.vec();
  pdl_begin();

  // -- the row's list ---------------------------------------------------------------------------
  float w = 0.0f, w_h = 0.0f;                     // gradient weights of the row
  if (MODE != kForward) {
    w = a.weight ? a.weight[r] : 0.0f;
    w_h = OP == kLogprob && a.weight_entropy ? a.weight_entropy[r] : 0.0f;
  }
  int target = -1;
  float x_target = 0.0f;
  if (OP == kLogprob && a.targets) {
    target = a.targets[r];
    if (target < -1 || target >= a.vocab) {
      if (tid == 0 && part == 0) raise(a.d_status, GSPARSE_DERR_INDEX_RANGE);
      target = -1;
    }
    if (target >= 0) x_target = Elem<T>::to(row.x[target]);
  }
  if (target < 0 && OP == kLogprob) w = 0.0f;
  double Q = 0.0, rho = 0.0;                      // mass of the list and what it leaves
  double list_max = 0.0, list_log = 0.0;          // renormalised list: maximum and log of the sum
  double w_list = 0.0, w_size = 0.0;              // sum of the alternatives' gradients; of the list's magnitudes
  const int nl = LIST ? (OP == kLogprob ? a.k + 1 : a.k) : 0;
  if constexpr (LIST) {
    ListShared& L = lp.list;
    if (OP == kTail || MODE != kForward) {
      for (int i = tid; i < kTable; i += B) L.table[i] = 0;
      for (int i = tid; i < kFilterWords; i += B) L.filter[i] = 0;
    }
    if (tid == 0) L.repeats = 0;
    float vmax = -INFINITY;
    for (int j = tid; j < nl; j += B) {
      int e;
      float v = 0.0f;
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
      L.x[j] = e >= 0 && (MODE != kBackward || row.owns(e)) ? Elem<T>::to(row.x[e]) : 0.0f;
      L.add[j] = v;
      if (e >= 0) vmax = fmaxf(vmax, v);
    }
    if (OP == kRenorm) list_max = (double)fmaxf(block_max(vmax, sh), kLowest);
    __syncthreads();
    double sum = 0.0, size = 0.0;
    for (int j = tid; j < nl; j += B) {
      const int e = L.idx[j];
      if (e < 0) continue;
      if (OP == kLogprob) {
        if (j > 0) sum += (double)L.add[j];
        size += fabs((double)L.add[j]);
      }
      else if (OP == kRenorm) sum += exp(((double)L.add[j] - list_max) * (double)a.it);
      else sum += exp((double)L.add[j]);
      if (OP == kTail || MODE != kForward)
        if (table_add(L, row.vec_of(e), row.lane_of(e))) L.repeats = 1;
    }
    block_sum2(sum, size, sh);
    if (OP == kLogprob) {
      w_list = sum;
      w_size = size;
    } else if (OP == kRenorm) {
      list_log = log(sum);
      Q = sum != 0.0 ? 1.0 : 0.0;                 // NaN in the list: Q = 1, the entries are NaN
      if (sum != sum) Q = sum;
    } else {
      Q = sum;
      rho = fmax(1.0 - sum, 0.0);
      if (sum != sum) rho = sum;
    }
  }

  // -- maximum and sums ----------------------------------------------------------------------------
  // Of the whole row; with kTail of the entries outside the list, whose sum as the difference of
  // two others would lose its digits when the list holds nearly all of the mass.
  float M = -INFINITY;
  double S = 0.0, Tt = 0.0;
  if (MODE != kBackward) {
    Running run;
    running_init(run);
    for (int i = row.v0 + tid; i < row.v1; i += U * B) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = i + u * B;
        v[u] = q < row.v1 ? __ldcg(vec + q) : make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
      }
      if constexpr (OP == kTail) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t mask = table_mask(lp.list, i + u * B + 1);
          if (mask) v[u] = masked<T>(v[u], mask);
        }
      }
      float high = run.m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[N];
        Elem<T>::unpack(v[u], x);
#pragma unroll
        for (int j = 0; j < N; ++j) high = fmaxf(high, x[j]);
      }
      if (high > run.m) running_raise(run, high, a.c);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[N];
        Elem<T>::unpack(v[u], x);
        running_add<N, ENT, FINE>(run, x, a);
      }
    }
    const int edge = row.edge(tid);
    if (edge >= 0) {
      float x[2] = {Elem<T>::to(row.x[edge]), -INFINITY};
      if constexpr (OP == kTail)
        if ((table_mask(lp.list, row.vec_of(edge)) >> row.lane_of(edge)) & 1u) x[0] = -INFINITY;
      if (x[0] > run.m) running_raise(run, x[0], a.c);
      running_add<2, ENT, FINE>(run, x, a);
    }
    const float mine = run.m;
    M = block_max(run.m, sh);
    running_raise(run, M, a.c);
    float s0, s1, t0, t1;
    unpair(run.s, &s0, &s1);
    unpair(run.t, &t0, &t1);
    S = (double)s0 + (double)s1;
    Tt = (double)t0 + (double)t1;
    block_sum2(S, Tt, sh);
    uint32_t kth = 0;
    if constexpr (TOP) kth = kth_key_of_block(order_key(mine), a.k);
    if (C > 1) {
      cg::cluster_group cl = cg::this_cluster();
      if (tid == 0) ex = Exchange{M, S, Tt, kth};
      cl.sync();
      float all = -INFINITY;
      for (int q = 0; q < C; ++q) {
        const Exchange* o = cl.map_shared_rank(&ex, q);
        all = fmaxf(all, o->m);
        kth = max(kth, o->kth);
      }
      S = Tt = 0.0;
      for (int q = 0; q < C; ++q) {
        const Exchange* o = cl.map_shared_rank(&ex, q);
        const float dd = max_nan((fmaxf(o->m, kLowest) - fmaxf(all, kLowest)) * a.c, -kFarBits);
        const double f = (double)ex2(dd);
        S += o->s * f;
        Tt += f * (o->t + (double)dd * o->s);
      }
      M = all;
    }

    // -- most likely tokens ----------------------------------------------------------------------
    // A thread's maximum is one entry, so the k-th largest of the threads' maxima is a lower bound of
    // the row's k-th largest entry; only threads whose maximum reaches it own candidates, and those
    // read their entries again (from L2).
    if constexpr (TOP) {
      TopShared& top = tp.top;
      if (tid == 0) top.count = 0;
      __syncthreads();
      const uint32_t bound = max(kth, kKeyNegInf + 1);
      const bool owner = order_key(mine) >= bound;
      uint32_t owners = __ballot_sync(kFull, owner);
      while (owners) {
        const int l = __ffs(owners) - 1;
        owners &= owners - 1;
        for (int i = row.v0 + (tid & ~31) + l + (tid & 31) * B; i < row.v1; i += 32 * B) {
          float x[N];
          Elem<T>::unpack(__ldcg(vec + i), x);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint32_t key = order_key(x[j]);
            if (key >= bound) cand_push(top, key, row.head + i * N + j);
          }
        }
      }
      if (owner && edge >= 0) {
        const uint32_t key = order_key(Elem<T>::to(row.x[edge]));
        if (key >= bound) cand_push(top, key, edge);
      }
      __syncthreads();
      bool again = top.count > kCand || !(S == S);
      if (C > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        if (part == 0) {
          int at = top.count;
          __syncthreads();
          for (int q = 1; q < C; ++q) {
            const TopShared* o = cl.map_shared_rank(&tp.top, q);
            const int n = o->count;
            if (n > kCand || at + n > kCand) again = true;
            if (again) break;
            for (int i = tid; i < n; i += B) top.cand[at + i] = o->cand[i];
            at += n;
          }
          if (tid == 0) top.count = at;
          __syncthreads();
        }
      }
      if (part == 0) {
        if (again) exact_top(row, a.k, kth, top, sh);
        const int n = top.count;
        // rank of a candidate = how many are larger; `per` neighbouring lanes share one
        int per = 1;
        while (per < 32 && 2 * per * n <= B) per *= 2;
        const double log_s = log(S);
        for (int base = 0; base < n; base += B / per) {
          const int i = base + tid / per;
          int above = 0;
          const unsigned long long me = i < n ? top.cand[i] : 0ull;
          for (int j = tid % per; j < n; j += per) above += top.cand[j] > me;
          for (int d = per >> 1; d > 0; d >>= 1) above += __shfl_xor_sync(kFull, above, d);
          if (i < n && tid % per == 0 && above < a.k) {
            const int e = (int)~(uint32_t)me;
            const int64_t o = (int64_t)r * a.k + above;
            a.top_idx[o] = e;
            a.top_val[o] = (float)(((double)Elem<T>::to(row.x[e]) - (double)M) * (double)a.it - log_s);
          }
        }
        for (int j = n + tid; j < a.k; j += B) {
          a.top_idx[(int64_t)r * a.k + j] = -1;
          a.top_val[(int64_t)r * a.k + j] = -INFINITY;
        }
      }
      // the row is read whole above: no gradient may be written before that is done
      if (C > 1) cg::this_cluster().sync();
    }
  }

  // -- statistics of the row, its loss -------------------------------------------------------------
  float ref = fmaxf(M, kLowest);                  // of the dense part of the gradient
  double S_dense = S;
  float ref_row = ref;                            // of the whole row
  double S_row = S;
  float ent = 0.0f;
  if (MODE == kBackward) {
    const float* st = a.stats_in + (int64_t)r * (OP == kTail ? 4 : 2);
    ref_row = ref = fmaxf(st[0], kLowest);
    S_row = S_dense = (double)st[1];
    if (OP == kTail) {
      ref = fmaxf(st[2], kLowest);
      S_dense = (double)st[3];
    }
    if (OP == kLogprob && a.weight_entropy) ent = a.entropy_in[r];
  }
  if constexpr (LIST && MODE != kBackward) {
    ListShared& L = lp.list;
    if (OP == kTail) {                            // the list's entries join the others'
      float high = -INFINITY;
      for (int j = tid; j < nl; j += B)
        if (L.idx[j] >= 0) high = fmaxf(high, L.x[j]);
      ref_row = fmaxf(fmaxf(block_max(high, sh), M), kLowest);
      double sum = 0.0, unused = 0.0;
      for (int j = tid; j < nl; j += B) {
        bool count = L.idx[j] >= 0;
        if (count && L.repeats)
          for (int i = 0; i < j; ++i) count = count && L.idx[i] != L.idx[j];
        if (count) sum += exp(((double)L.x[j] - (double)ref_row) * (double)a.it);
      }
      block_sum2(sum, unused, sh);
      S_row = sum + (S != 0.0 ? S * exp(((double)ref - (double)ref_row) * (double)a.it) : 0.0);
    }
    if (OP == kTail && S_dense == 0.0) rho = 0.0; // no entry is left for the rest
    double loss = 0.0, unused = 0.0;
    const double log_s = log(S_row);
    for (int j = tid; j < nl; j += B) {
      if (L.idx[j] < 0 || Q == 0.0) continue;
      const double lq = OP == kRenorm ? ((double)L.add[j] - list_max) * (double)a.it - list_log : (double)L.add[j];
      const double q = exp(lq);
      const double lp_j = S_row == 0.0 ? -(double)INFINITY : ((double)L.x[j] - (double)ref_row) * (double)a.it - log_s;
      if (!(q == 0.0)) loss += q * (lq - lp_j);
    }
    block_sum2(loss, unused, sh);
    if (!(rho == 0.0))
      loss += rho * (log(rho) - (((double)ref - (double)ref_row) * (double)a.it + log(S_dense) - log_s));
    if (Q == 0.0 && rho == 0.0) loss = 0.0;
    if (part == 0 && tid == 0) {
      a.out[r] = (float)loss;
      if (a.stats) {
        float* st = a.stats + (int64_t)r * (OP == kTail ? 4 : 2);
        st[0] = ref_row;
        st[1] = (float)S_row;
        if (OP == kTail) {
          st[2] = ref;
          st[3] = (float)S_dense;
        }
      }
    }
  }
  if (OP == kTail && MODE == kBackward && S_dense == 0.0) rho = 0.0;
  if (OP == kLogprob && MODE != kBackward) {
    const double log_s = log(S);
    const bool nothing = S == 0.0;
    ent = nothing ? 0.0f : (float)(log_s - 0.6931471805599453 * (Tt / S));
    if (part == 0 && tid == 0) {
      if (a.out)
        a.out[r] = target < 0 ? 0.0f
                   : nothing  ? -INFINITY
                              : (float)(((double)x_target - (double)M) * (double)a.it - log_s);
      if (a.entropy) a.entropy[r] = ent;
      if (a.stats) {
        a.stats[2 * (int64_t)r] = ref;
        a.stats[2 * (int64_t)r + 1] = (float)S;
      }
    }
  }

  // the others may still read this CTA's shared memory
  if (MODE == kForward && !TOP && C > 1) cg::this_cluster().sync();

  // -- gradient ----------------------------------------------------------------------------------
  if constexpr (MODE != kForward) {
    // dense: g = p (A + Bl log2 p), p = 2^((x - ref) c - l2)
    float A, Bl = 0.0f, A_list;
    if (OP == kLogprob) {
      A = (float)(-(double)a.it * ((double)w + w_list + (double)w_h * (double)ent));
      Bl = -a.it * w_h * 0.69314718f;
      A_list = A;
    } else if (OP == kRenorm) {
      A_list = A = (float)((double)a.it * (double)w * Q);
    } else {
      const double R = S_dense != 0.0 ? S_dense / S_row * exp(((double)ref - (double)ref_row) * (double)a.it) : 0.0;
      A_list = (float)((double)a.it * (double)w * (Q + rho));
      A = (float)((double)a.it * (double)w * ((Q + rho) * R - rho));
    }
    const bool nothing = S_row == 0.0;            // nothing but -inf: no distribution, no gradient
    if (nothing) A = A_list = Bl = 0.0f;
    const float l2 = S_dense == 0.0 ? 0.0f : (float)log2(S_dense);
    // no weight: zeros, whatever the row holds
    const bool none = OP == kLogprob ? (w == 0.0f && w_h == 0.0f && w_size == 0.0) : w == 0.0f;
    T* dx = static_cast<T*>(a.dlogits) + (int64_t)r * a.dstride;
    if (C > 1 && MODE == kFused) {
      if (!TOP) cg::this_cluster().sync();        // every CTA has read the list's and target's entries
    } else {
      __syncthreads();
    }
    if (none) A = Bl = 0.0f;
    const f2 nref = pair(-ref, -ref), c2 = pair(a.c, a.c), nl2 = pair(-l2, -l2), A2 = pair(A, A), B2 = pair(Bl, Bl);
    auto grad = [&](float* x, int n) {
#pragma unroll
      for (int i = 0; i < n; i += 2) {
        float d0, d1;
        unpair(add2(pair(x[i], x[i + 1]), nref), &d0, &d1);
        const f2 d = pair(max_nan(d0, -a.far), max_nan(d1, -a.far));
        const f2 q = fma2(d, c2, nl2);
        float q0, q1;
        unpair(q, &q0, &q1);
        const f2 p = pair(ex2(q0), ex2(q1));
        const f2 g = OP == kLogprob ? mul2(p, fma2(q, B2, A2)) : mul2(p, A2);
        unpair(g, &x[i], &x[i + 1]);
      }
    };
    if (((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(row.x)) & 15u) == 0) {
      uint4* dvec = reinterpret_cast<uint4*>(dx + row.head);
      for (int i = row.v0 + tid; i < row.v1; i += U * B) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = i + u * B;
          if (q < row.v1 && !none) v[u] = __ldcs(vec + q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int q = i + u * B;
          if (q >= row.v1) break;
          float x[N];
          if (none) {
            v[u] = make_uint4(0, 0, 0, 0);
          } else {
            Elem<T>::unpack(v[u], x);
            grad(x, N);
            v[u] = Elem<T>::pack(x);
          }
          __stcs(dvec + q, v[u]);
        }
      }
    } else {                                      // rows that start at different offsets from 16 bytes
      for (int e = row.head + row.v0 * N + tid; e < row.head + row.v1 * N; e += B) {
        float x[2] = {none ? 0.0f : Elem<T>::to(row.x[e]), -INFINITY};
        if (!none) grad(x, 2);
        dx[e] = Elem<T>::from(x[0]);
      }
    }
    const int edge = row.edge(tid);
    if (edge >= 0) {
      float x[2] = {none ? 0.0f : Elem<T>::to(row.x[edge]), -INFINITY};
      if (!none) grad(x, 2);
      dx[edge] = Elem<T>::from(x[0]);
    }
    __syncthreads();
    // the list's entries, over what the dense part wrote there
    if (none || nothing) return;
    auto value = [&](float x, double add) {
      const double lp2 = ((double)x - (double)ref_row) * (double)a.it - log(S_row);
      const double p = exp(lp2);
      double g = p * (double)A_list + add;
      if (OP == kLogprob && Bl != 0.0f && p != 0.0) g -= (double)a.it * (double)w_h * p * lp2;
      return (float)g;
    };
    if constexpr (LIST) {
      ListShared& L = lp.list;
      for (int j = tid; j < nl; j += B) {
        const int e = L.idx[j];
        if (e < 0 || !row.owns(e)) continue;
        double add = 0.0;
        bool mine = true;
        for (int i = L.repeats ? 0 : j; i < (L.repeats ? nl : j + 1); ++i) {
          if (L.idx[i] != e) continue;
          if (i < j) mine = false;
          if (OP == kLogprob) add += (double)a.it * (double)L.add[i];
          else if (Q != 0.0) {
            const double lq = OP == kRenorm ? ((double)L.add[i] - list_max) * (double)a.it - list_log : (double)L.add[i];
            add -= (double)a.it * (double)w * exp(lq);
          }
        }
        if (mine) dx[e] = Elem<T>::from(value(L.x[j], add));
      }
    } else {
      if (tid == 0 && target >= 0 && row.owns(target))
        dx[target] = Elem<T>::from(value(x_target, (double)a.it * (double)w));
    }
  }
}

// ---- launch -----------------------------------------------------------------------------------------

template <class T, int OP, bool TOP, int MODE>
int voc_launch(const VocArgs& a, int threads, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * a.split));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE != kBackward && a.split > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, voc_kernel<T, OP, TOP, MODE>, a) != cudaSuccess) {
    cudaGetLastError();
    return GSPARSE_ERR_CUDA;
  }
  return launch_status();
}

template <int OP, bool TOP, int MODE>
int voc_by_type(int32_t dtype, VocArgs a, cudaStream_t st) {
  const int n = dtype == GSPARSE_F32 ? 4 : 8;
  const int64_t nv = cdiv(a.vocab, n);
  // few rows: split each over up to 8 CTAs, as long as a CTA keeps 512 vectors
  int split = 1;
  while (split < 8 && (int64_t)a.rows * split < 2 * sm_count() && nv / (2 * split) >= 512) split *= 2;
  a.split = split;
  int threads = 64;
  while (threads < kVocThreads && (int64_t)threads * kVocUnroll * split < nv) threads *= 2;
  if (TOP) while (threads < kVocThreads && threads < 2 * a.k) threads *= 2;
  if (dtype == GSPARSE_F32) return voc_launch<float, OP, TOP, MODE>(a, threads, st);
  if (dtype == GSPARSE_BF16) return voc_launch<__nv_bfloat16, OP, TOP, MODE>(a, threads, st);
  return voc_launch<__half, OP, TOP, MODE>(a, threads, st);
}

bool voc_dtype(int32_t t) { return t == GSPARSE_F32 || t == GSPARSE_BF16 || t == GSPARSE_F16; }

// Arguments common to the four calls.
int voc_common(VocArgs& a, const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t stride,
               float inv_temperature, void* dlogits, int64_t dstride, int32_t* d_status) {
  if (!voc_dtype(dtype) || rows < 0 || vocab < 1 || stride < 0) return GSPARSE_ERR_INVALID_ARG;
  if (!(inv_temperature > 0.0f) || !isfinite(inv_temperature)) return GSPARSE_ERR_INVALID_ARG;
  if (rows > INT32_MAX / 8 || vocab > GSPARSE_MAX_VOCAB) return GSPARSE_ERR_UNSUPPORTED;
  const uintptr_t align = dtype == GSPARSE_F32 ? 3 : 1;
  if (rows > 0 && !logits) return GSPARSE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & align) || (reinterpret_cast<uintptr_t>(dlogits) & align))
    return GSPARSE_ERR_INVALID_ARG;
  if (dlogits && rows > 1 && dstride < vocab) return GSPARSE_ERR_INVALID_ARG;
  if (dlogits == logits && dlogits && rows > 1 && dstride != stride) return GSPARSE_ERR_INVALID_ARG;
  const double c = (double)inv_temperature * 1.4426950408889634;
  a.c = (float)c;
  a.c_lo = (float)(c - (double)a.c);
  a.far = kFarBits / a.c;
  if (!isfinite(a.c) || !isfinite(a.far) || a.far == 0.0f) return GSPARSE_ERR_UNSUPPORTED;
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
  if (dlogits)
    return top_k ? voc_by_type<kLogprob, true, kFused>(dtype, a, s) : voc_by_type<kLogprob, false, kFused>(dtype, a, s);
  return top_k ? voc_by_type<kLogprob, true, kForward>(dtype, a, s) : voc_by_type<kLogprob, false, kForward>(dtype, a, s);
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
  return voc_by_type<kLogprob, false, kBackward>(dtype, a, (cudaStream_t)stream);
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
    return dlogits ? voc_by_type<kTail, false, kFused>(dtype, a, s) : voc_by_type<kTail, false, kForward>(dtype, a, s);
  return dlogits ? voc_by_type<kRenorm, false, kFused>(dtype, a, s) : voc_by_type<kRenorm, false, kForward>(dtype, a, s);
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
  if (mode == GSPARSE_DISTILL_TAIL) return voc_by_type<kTail, false, kBackward>(dtype, a, (cudaStream_t)stream);
  return voc_by_type<kRenorm, false, kBackward>(dtype, a, (cudaStream_t)stream);
}

}  // extern "C"

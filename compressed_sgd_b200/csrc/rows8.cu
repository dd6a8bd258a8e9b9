// Rows in 8 bits with one scale each, the root-mean-square norm that writes them, and its gradient.
//
// A row's scale is a power of two, 2^e with the smallest e from -126 to 121 for which no entry exceeds 127 * 2^e: the value q * 2^e has
// seven bits, so bf16 holds it exactly and the products that read it (linear8.cu) lose nothing to a conversion. Against a
// scale of max / 127 the step is up to twice as wide, 1.44 times on average.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"

namespace gs {
namespace {

constexpr int kRowsPerBlock = 4;     // rows of a block whose rows take one warp each
constexpr int kMostThreads = 1024;

template <class T> struct Type;
template <> struct Type<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Type<__nv_bfloat16> {
  static constexpr int N = 8;
  using Two = __nv_bfloat162;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ float2 get(Two v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ Two put(float a, float b) { return __floats2bfloat162_rn(a, b); }
};
template <> struct Type<__half> {
  static constexpr int N = 8;
  using Two = __half2;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ float2 get(Two v) { return __half22float2(v); }
  static __device__ __forceinline__ Two put(float a, float b) { return __floats2half2_rn(a, b); }
};

// How a row's entries are shared out. kVectors: every row starts at a 16-byte boundary and is whole vectors. kShifted: rows start
// anywhere, but all matrices' rows at the same place between two boundaries; vectors lie between boundaries, those at the row's ends
// are read and written entry by entry. Rows in 8 bits start at boundaries of their own, so a group of their bytes takes a vector's end
// and the next one's start: a warp takes 31 vectors, and its last lane holds the next warp's first once more, for its bytes.
// kEntries: rows of any alignment, entry by entry. kWords: whole rows of four bytes at a time. kWide: whole rows of 32 bytes at a time,
// from 32-byte boundaries (half the accesses and addresses of kVectors: 8192 x 8192 fp32 with the norm, 166 us; 175).
enum { kVectors, kShifted, kEntries, kWords, kWide };

__device__ __forceinline__ void load_wide(uint32_t* v, const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_wide(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int V> struct Constant { static constexpr int value = V; };

// A thread's E entries of a row of `depth`, vector after vector (entry after entry), thread after thread. `off`: the row's start
// behind a boundary, in entries (kShifted only).
template <class T, int MODE, int E>
struct Mine {
  static constexpr int N = MODE == kEntries ? 1 : MODE == kWords ? 4 / (int)sizeof(T) : MODE == kWide ? 2 * Type<T>::N : Type<T>::N;
  int tid, threads, depth, off;

  __device__ __forceinline__ int first(int j) const {
    if constexpr (MODE == kShifted) return (j * (threads / 32 * 31) + tid - (tid >> 5)) * N - off;
    return (j * threads + tid) * N;
  }
  // Whether this thread's entries are its own, and not the next warp's.
  __device__ __forceinline__ bool own() const { return MODE != kShifted || (tid & 31) < 31; }
  __device__ __forceinline__ bool whole(int at) const { return MODE == kShifted ? at >= 0 && at + N <= depth : at < depth; }
  __device__ __forceinline__ bool none(int at) const { return at >= depth || (MODE == kShifted && at + N <= 0); }
  __device__ __forceinline__ bool in(int at) const { return at < depth && (MODE != kShifted || at >= 0); }

  // As they lie in memory, and as numbers.
  union Raw {
    uint4 vec[E * sizeof(T) / 16];
    uint32_t word[E * sizeof(T) / 4];
    T one[E];
    __device__ __forceinline__ Raw() {}
  };

  __device__ __forceinline__ void fetch(Raw& raw, const T* row) const {
#pragma unroll
    for (int j = 0; j < E / N; ++j) {
      const int at = first(j);
      if constexpr (MODE == kEntries) {
        raw.one[j] = at < depth ? row[at] : Type<T>::put(0.0f);
      } else if constexpr (MODE == kWords) {
        raw.word[j] = at < depth ? *reinterpret_cast<const uint32_t*>(row + at) : 0u;
      } else if constexpr (MODE == kWide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw.word[j * 8 + i] = 0u;
        if (at < depth) load_wide(raw.word + j * 8, row + at);
      } else {
        raw.vec[j] = make_uint4(0, 0, 0, 0);
        if (whole(at)) raw.vec[j] = *reinterpret_cast<const uint4*>(row + at);
        else if (MODE == kShifted && !none(at)) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (in(at + i)) raw.one[j * N + i] = row[at + i];
        }
      }
    }
  }

  static __device__ __forceinline__ void numbers(float (&v)[E], const Raw& raw) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 f = Type<T>::get(*reinterpret_cast<const typename Type<T>::Two*>(raw.one + i));
        v[i] = f.x;
        v[i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = raw.one[i];
    }
  }

  static __device__ __forceinline__ void held(Raw& raw, const float (&v)[E]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < E; i += 2) *reinterpret_cast<typename Type<T>::Two*>(raw.one + i) = Type<T>::put(v[i], v[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) raw.one[i] = v[i];
    }
  }

  __device__ __forceinline__ void write(T* row, const Raw& raw) const {
    if (!own()) return;
#pragma unroll
    for (int j = 0; j < E / N; ++j) {
      const int at = first(j);
      if constexpr (MODE == kEntries) {
        if (at < depth) row[at] = raw.one[j];
      } else if constexpr (MODE == kWords) {
        if (at < depth) *reinterpret_cast<uint32_t*>(row + at) = raw.word[j];
      } else if constexpr (MODE == kWide) {
        if (at < depth) store_wide(row + at, raw.word + j * 8);
      } else {
        if (whole(at)) *reinterpret_cast<uint4*>(row + at) = raw.vec[j];
        else if (MODE == kShifted && !none(at)) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (in(at + i)) row[at + i] = raw.one[j * N + i];
        }
      }
    }
  }

  __device__ __forceinline__ void load(float (&v)[E], const T* row) const {
    Raw raw;
    fetch(raw, row);
    numbers(v, raw);
  }

  __device__ __forceinline__ void store(T* row, const float (&v)[E]) const {
    Raw raw;
    held(raw, v);
    write(row, raw);
  }

  // N entries of 16 bits; with kVectors they start at a multiple of their own size.
  template <class W>
  __device__ __forceinline__ void narrow(float* v, const W* w, int at) const {
    W e[N];
    if constexpr (MODE == kWide && N == 16) load_wide(reinterpret_cast<uint32_t*>(e), w + at);
    else if constexpr (MODE == kWide || (MODE == kVectors && N == 8)) *reinterpret_cast<uint4*>(e) = __ldg(reinterpret_cast<const uint4*>(w + at));
    else if constexpr (MODE == kVectors) *reinterpret_cast<uint2*>(e) = __ldg(reinterpret_cast<const uint2*>(w + at));
    else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = in(at + i) ? w[at + i] : Type<W>::put(0.0f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Type<W>::get(e[i]);
  }

  // Entries of fp32, bf16 or fp16, whatever T is (the norm's weight).
  __device__ __forceinline__ void load_any(float (&v)[E], const void* p, int dtype) const {
#pragma unroll
    for (int j = 0; j < E / N; ++j) {
      const int at = first(j);
#pragma unroll
      for (int i = 0; i < N; ++i) v[j * N + i] = 0.0f;
      if (none(at)) continue;
      if (dtype == GSPARSE_F32) {
        const float* w = static_cast<const float*>(p);
        if constexpr (MODE == kWide) {
#pragma unroll
          for (int i = 0; i < N; i += 8) load_wide(reinterpret_cast<uint32_t*>(v + j * N + i), w + at + i);
        } else if constexpr (MODE == kVectors) {
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(w + at + i));
            v[j * N + i] = f.x; v[j * N + i + 1] = f.y; v[j * N + i + 2] = f.z; v[j * N + i + 3] = f.w;
          }
        } else if (MODE == kShifted && fours_within(at, N, depth) && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
          // N floats from anywhere out of whole vectors; the place is the row's
          float f[N + 4];
          const int d = at & 3;
#pragma unroll
          for (int i = 0; i < N + 4; i += 4) *reinterpret_cast<float4*>(f + i) = __ldg(reinterpret_cast<const float4*>(w + at - d + i));
          auto take = [&](auto from) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[j * N + i] = f[i + decltype(from)::value];
          };
          if (d == 0) take(Constant<0>());
          else if (d == 1) take(Constant<1>());
          else if (d == 2) take(Constant<2>());
          else take(Constant<3>());
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) v[j * N + i] = in(at + i) ? w[at + i] : 0.0f;
        }
      } else if (dtype == GSPARSE_BF16) {
        narrow(&v[j * N], static_cast<const __nv_bfloat16*>(p), at);
      } else {
        narrow(&v[j * N], static_cast<const __half*>(p), at);
      }
    }
  }

  // The entries' low bytes (of y's bits) into a row in 8 bits, which starts at a 16-byte boundary; zeros where not `fine`.
  __device__ __forceinline__ void bytes(int8_t* out, const float (&y)[E], bool fine) const {
#pragma unroll
    for (int j = 0; j < E / N; ++j) {
      const int at = first(j);
      const float* s = y + j * N;
      auto four = [&](int i) {
        const uint32_t a01 = __byte_perm(__float_as_uint(s[i]), __float_as_uint(s[i + 1]), 0x0040);
        const uint32_t a23 = __byte_perm(__float_as_uint(s[i + 2]), __float_as_uint(s[i + 3]), 0x0040);
        return fine ? __byte_perm(a01, a23, 0x5410) : 0u;
      };
      if constexpr (MODE == kEntries) {
        if (at < depth) out[at] = fine ? (int8_t)__float_as_uint(s[0]) : 0;
      } else if constexpr (MODE == kWide) {
        if (at >= depth) continue;
        if constexpr (N == 16) *reinterpret_cast<uint4*>(out + at) = make_uint4(four(0), four(4), four(8), four(12));
        else *reinterpret_cast<uint2*>(out + at) = make_uint2(four(0), four(4));
      } else if constexpr (MODE == kVectors) {
        if (at >= depth) continue;
        if constexpr (N == 8) *reinterpret_cast<uint2*>(out + at) = make_uint2(four(0), four(4));
        else *reinterpret_cast<uint32_t*>(out + at) = four(0);
      } else {
        const uint64_t mine = N == 8 ? (uint64_t)four(0) | (uint64_t)four(N == 8 ? 4 : 0) << 32 : four(0);
        const uint64_t next = N == 8 ? __shfl_down_sync(kFull, (unsigned long long)mine, 1) : __shfl_down_sync(kFull, (uint32_t)mine, 1);
        const uint64_t both = mine >> (8 * off) | (off ? next << (8 * (N - off)) : 0);
        const int group = at + off;
        if (!own() || group >= depth) continue;    // (after the exchange)
        if (group + N <= depth) {
          if constexpr (N == 8) *reinterpret_cast<uint64_t*>(out + group) = both;
          else *reinterpret_cast<uint32_t*>(out + group) = (uint32_t)both;
        } else {
          for (int i = 0; group + i < depth; ++i) out[group + i] = (int8_t)(both >> (8 * i));
        }
      }
    }
  }
};

struct RowArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* h;
  void* y;
  int8_t* q;
  float* scale;
  float* rstd;
  int64_t rows, x_stride, residual_stride, h_stride, y_stride, q_stride;
  double inv_depth;
  int depth, weight_dtype, warps;   // warps of a row
  float eps;
};

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float power(int e) { return __int_as_float((e + 127) << 23); }

constexpr uint32_t kScaleBorder = 0x7e0000u;       // the significand's bits of 127 * 2^e

// The exponent of the scale of a row whose largest magnitude has these (finite) bits.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  // top = m 2^(k - 127) with 1 <= m < 2: 127 / 64 is the border of m. What is below 2^-119 takes the smallest scale.
  const int k = (int)(top >> 23);
  const int e = k - 127 - 6 + ((top & 0x7fffffu) > kScaleBorder ? 1 : 0);
  return e < -126 ? -126 : e > 121 ? 121 : e;     // 121: 64 * 2^122 is no fp32 number
}

// (ms)^(-1/2): two steps of Newton's iteration from the fp32 value, 2^-22 -> 2^-43 -> 2^-52 or so.
__device__ __forceinline__ double inverse_root(double ms) {
  if (!(ms < 0x1p100)) return 1.0 / sqrt(ms);      // beyond fp32, infinite, NaN (from below eps keeps it off)
  double r = (double)rsqrtf((float)ms);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __fma_rn(0.5 * r, __fma_rn(-ms * r, r, 1.0), r);
  return r;
}

// The larger one, NaN where one is.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kRound = 12582912.0f;              // 1.5 * 2^23: adding it rounds to an integer, held in the low bits

// v r w in two parts, good to about 2^-45 of it where far_off (below) is false.
__device__ __forceinline__ float2 in_parts(float v, float r_hi, float r_lo, float w) {
  const float rw = __fmul_rn(r_hi, w);
  const float rw_lo = __fmaf_rn(r_lo, w, __fmaf_rn(r_hi, w, -rw));
  const float hi = __fmul_rn(v, rw);
  return make_float2(hi, __fmaf_rn(v, rw_lo, __fmaf_rn(v, rw, -hi)));
}

// An entry's number of steps, v r w / 2^e, rounded: what the formula gives in 64 bits.
__device__ __forceinline__ float steps_of(float v, float r_hi, float r_lo, float w, float up) {
  const float2 y = in_parts(v, r_hi, r_lo, w);
  const float t = y.x * up, lo = y.y;
  const float m = t + kRound, f = t - (m - kRound);          // within a half, exact
  // past a half with the small part? The distances to it are exact, so the signs of these sums are.
  return m + (__fmaf_rn(lo, up, f - 0.5f) > 0.0f ? 1.0f : __fmaf_rn(lo, up, f + 0.5f) < 0.0f ? -1.0f : 0.0f);
}

// Rows whose r or whose entries' r v would leave the second part of in_parts (or even r w itself) below fp32's smallest steps: in 64
// bits, entry by entry, from h as it was written or summed again. Kept apart and last, over what the others' way has written, so that
// other rows pay for two comparisons (8192 x 4096 bf16 with the residual: 70.8 us with the reading back, 70.5 without). With ms the
// mean square, such rows have ms + eps beyond 2^+-48 or ms below 2^-60 of it; for the others and weights of magnitudes from 2^-64 to 2^64,
// r w is at least 2^-88 and the entries that have steps at all (2^-8 of the largest) at least 2^-102, whose last bits in two parts
// (2^-45 of them) are 2^-147: fp32 still has those. Rows of zeros stay with the others.
__device__ __forceinline__ bool far_off(double ms, double eps) {
  const double t = ms + eps;
  return ms > 0.0 && t < 0x1p1000 && !(t >= 0x1p-48 && t <= 0x1p48 && ms >= t * 0x1p-60);
}

template <class T>
__device__ __noinline__ void far_row(const RowArgs& a, int64_t row, double r, int tid, double* tops) {
  const int threads = a.warps * 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool one = a.warps == 1;
  if (one) __syncwarp();
  else __syncthreads();                            // h, y and q are written, and the sums in `tops` have been read
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* residual = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  const T* h = a.h ? static_cast<const T*>(a.h) + row * a.h_stride : nullptr;
  auto y_of = [&](int k) {
    const float v = h ? Type<T>::get(h[k]) : residual ? Type<T>::get(Type<T>::put(Type<T>::get(x[k]) + Type<T>::get(residual[k]))) : Type<T>::get(x[k]);
    const float w = a.weight_dtype == GSPARSE_F32    ? static_cast<const float*>(a.weight)[k]
                    : a.weight_dtype == GSPARSE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.weight)[k])
                                                     : __half2float(static_cast<const __half*>(a.weight)[k]);
    return (double)v * r * (double)w;
  };
  const double infinite = __longlong_as_double(0x7ff0000000000000ll);
  double top = 0.0;
  for (int k = tid; k < a.depth; k += threads) {
    const double y = y_of(k);
    if (a.y) static_cast<T*>(a.y)[row * a.y_stride + k] = Type<T>::put((float)y);
    top = fabs(y) < infinite ? fmax(top, fabs(y)) : infinite;  // (NaN too)
  }
  if (!a.q) return;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, d));
  if (!one) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = lane < a.warps ? tops[lane] : 0.0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, d));
  }
  const bool fine = top < infinite;
  // as scale_exponent, of a number of 64 bits
  const long long bits = __double_as_longlong(top);
  int e = (int)(bits >> 52) - 1023 - 6 + ((bits & 0xfffffffffffffll) > ((long long)kScaleBorder << 29) ? 1 : 0);
  e = !fine ? 0 : e < -126 ? -126 : e > 121 ? 121 : e;
  if (tid == 0) a.scale[row] = fine ? power(e) : __int_as_float(0x7fc00000);
  const double up = __longlong_as_double((long long)(1023 - e) << 52);
  int8_t* q = a.q + row * a.q_stride;
  for (int k = tid; k < a.depth; k += threads) q[k] = fine ? (int8_t)__double2int_rn(fmin(fmax(y_of(k) * up, -127.0), 127.0)) : 0;
}

// One pass over the rows: the sum with the residual, the norm, the 8 bits. A row stays in its threads' registers.
//
// An entry's steps t come from three fp32 roundings, so they are off by less than 2^-15: only those that lie closer than 2^-14 to
// the middle between two integers (one of 2^13) are worked out again in two parts. All of them in two parts, with divisions and roots in
// 64 bits: 92 against 52 us for 8192 x 4096 bf16 with the residual (235 MB, 36 us at the measured copy bandwidth).
template <class T, int MODE, int E, bool NORM, int MOST>
__global__ void __launch_bounds__(MOST, MODE == kEntries ? 1 : MOST == 384 ? 3 : MOST == 512 ? 2 : 1) rows_kernel(const __grid_constant__ RowArgs a) {
  pdl_begin();
  __shared__ double sums[kMostThreads / 32];
  __shared__ uint32_t tops[kMostThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool one = a.warps == 1;
  const int64_t row = one ? (int64_t)blockIdx.x * kRowsPerBlock + warp : blockIdx.x;
  if (row >= a.rows) return;                       // whole warps, and only where no barrier follows
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  using M = Mine<T, MODE, E>;
  const M mine{one ? lane : (int)threadIdx.x, a.warps * 32, a.depth,
               MODE == kShifted ? (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)) : 0};
  typename M::Raw raw;                             // h
  float v[E], y[E];
  mine.fetch(raw, x);
  float r_hi = 1.0f, r_lo = 0.0f;
  bool far = false;
  if constexpr (NORM) {
    if (a.residual) {
      mine.load(y, static_cast<const T*>(a.residual) + row * a.residual_stride);
      M::numbers(v, raw);
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] += y[i];
      M::held(raw, v);
    }
    if (a.h) mine.write(static_cast<T*>(a.h) + row * a.h_stride, raw);
    mine.load_any(y, a.weight, a.weight_dtype);
    M::numbers(v, raw);
    // squares of any size, and a sum that is good to the last of them: 64 bits
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < E; ++i) ss = __fma_rn((double)v[i], (double)v[i], ss);
    ss = warp_sum(mine.own() ? ss : 0.0);
    if (!one) {
      if (lane == 0) sums[warp] = ss;
      __syncthreads();
      ss = lane < a.warps ? sums[lane] : 0.0;
      ss = warp_sum(ss);
    }
    const double ms = ss * a.inv_depth, r = inverse_root(ms + (double)a.eps);
    r_hi = (float)r;
    r_lo = (float)(r - (double)r_hi);
    if (a.rstd && mine.tid == 0) a.rstd[row] = r_hi;
    far = far_off(ms, (double)a.eps);
    if (far) {                                     // kept for far_row: r is at least 2^-128 here, and r 2^32 has a second part
      r_hi = (float)(r * 0x1p32);
      r_lo = (float)(r * 0x1p32 - (double)r_hi);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = v[i] * (r_hi * y[i]);
    if (a.y) {
      float w[E];
      mine.load_any(w, a.weight, a.weight_dtype);
#pragma unroll
      for (int i = 0; i < E; ++i) {                // in two parts: rounded once
        const float rw = __fmul_rn(r_hi, w[i]);
        w[i] = __fmaf_rn(v[i], rw, v[i] * __fmaf_rn(r_lo, w[i], __fmaf_rn(r_hi, w[i], -rw)));
      }
      mine.store(static_cast<T*>(a.y) + row * a.y_stride, w);
    }
    if (!a.q) {
      if (far) far_row<T>(a, row, ((double)r_hi + (double)r_lo) * 0x1p-32, mine.tid, sums);
      return;
    }
  } else {
    M::numbers(y, raw);
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) top = larger(top, fabsf(y[i]));
  uint32_t bits = __reduce_max_sync(kFull, mag_key(top));    // NaN above the infinities above the numbers
  if (!one) {
    if (lane == 0) tops[warp] = bits;
    __syncthreads();
    bits = __reduce_max_sync(kFull, lane < a.warps ? tops[lane] : 0u);
  }
  const bool fine = bits < 0x7f800000u;            // no infinity, no NaN
  if constexpr (NORM) {
    // The largest entry at the border between two scales, up to its roundings: whether one is above it, in two parts.
    if (fine && (bits & 0x7fffffu) - (kScaleBorder - 4) <= 8u) {
      const uint32_t at = (bits & 0x7f800000u) | kScaleBorder;
      const float border = __uint_as_float(at);
      float w[E];
      mine.load_any(w, a.weight, a.weight_dtype);
      mine.numbers(v, raw);
      bool over = false;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float2 p = in_parts(fabsf(v[i]), r_hi, r_lo, fabsf(w[i]));
        over = over || (p.x - border) + p.y > 0.0f;            // (of entries near the border the difference is exact)
      }
      over = one ? __any_sync(kFull, over) : __syncthreads_or(over);
      bits = at + (over ? 1u : 0u);
    }
  }
  const int e = fine ? scale_exponent(bits) : 0;
  const float up = power(-e);                      // -121 <= -e <= 126
  if (mine.tid == 0) a.scale[row] = fine ? power(e) : __int_as_float(0x7fc00000);
  float near = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float t = y[i] * up;                     // at most 127 and a rounding
    y[i] = t + kRound;
    if constexpr (NORM) near = fmaxf(near, fabsf(t - (y[i] - kRound)));
  }
  if constexpr (NORM) {
    if (near > 0.5f - 0x1p-14f && fine) {
      M::numbers(v, raw);
      float w[E];
      mine.load_any(w, a.weight, a.weight_dtype);
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = steps_of(v[i], r_hi, r_lo, w[i], up);
    }
  }
  if (e == 121) {                                  // where entries may be above 127 * 2^121
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = fminf(fmaxf(y[i], kRound - 127.0f), kRound + 127.0f);
  }
  mine.bytes(a.q + row * a.q_stride, y, fine);
  if constexpr (NORM) {
    if (far) far_row<T>(a, row, ((double)r_hi + (double)r_lo) * 0x1p-32, mine.tid, sums);
  }
}

// ---- read back ------------------------------------------------------------------------------------------

// Rows of `out` that start at 16-byte boundaries: 16 entries a thread.
template <class T>
__global__ void __launch_bounds__(256) dequant_kernel(const int8_t* q, int64_t q_stride, const float* scale, int64_t rows, int depth,
                                                      T* out, int64_t out_stride) {
  pdl_begin();
  const int64_t per = (depth + 15) / 16, all = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / per;
    const int at = (int)(i - row * per) * 16;
    const float s = __ldg(scale + row);
    const int8_t* p = q + row * q_stride + at;
    T* o = out + row * out_stride + at;
    const int left = depth - at;
    if (left >= 16) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p));
      const int8_t* b = reinterpret_cast<const int8_t*>(&raw);
      union { uint4 vec[sizeof(T)]; T one[16]; } e;
#pragma unroll
      for (int k = 0; k < 16; ++k) e.one[k] = Type<T>::put((float)b[k] * s);
#pragma unroll
      for (int k = 0; k < (int)sizeof(T); ++k) reinterpret_cast<uint4*>(o)[k] = e.vec[k];
    } else {
      for (int k = 0; k < left; ++k) o[k] = Type<T>::put((float)p[k] * s);
    }
  }
}

// Rows of any alignment. A thread makes the vectors of 16 bytes of `out` between two boundaries, from the row's N bytes that they stand for: with rows that
// start off a boundary those are parts of two groups of N.
template <class T>
__global__ void __launch_bounds__(256) dequant_shifted_kernel(const int8_t* q, int64_t q_stride, const float* scale, int64_t rows, int depth,
                                                              T* out, int64_t out_stride, int per) {
  pdl_begin();
  constexpr int N = Type<T>::N;
  const int64_t all = rows * per, step = (int64_t)gridDim.x * blockDim.x;
  int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= all) return;
  // (a division once; the steps after it add up)
  const int64_t step_rows = step / per;
  const int step_at = (int)(step - step_rows * per);
  int64_t row = i / per;
  int v = (int)(i - row * per);
  for (; i < all; i += step) {
    T* to = out + row * out_stride;
    const int8_t* from = q + row * q_stride;
    const float s = __ldg(scale + row);
    const int off = (int)((reinterpret_cast<uintptr_t>(to) & 15) / sizeof(T)), at = v * N - off;
    auto group = [&](int g) -> uint64_t {          // bytes [g, g + N) of the row, 0 where it has none; g a multiple of N
      if (g < 0 || g >= depth) return 0;
      if (g + N <= depth) {
        if constexpr (N == 8) return __ldg(reinterpret_cast<const unsigned long long*>(from + g));
        else return __ldg(reinterpret_cast<const uint32_t*>(from + g));
      }
      uint64_t b = 0;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (g + k < depth) b |= (uint64_t)(uint8_t)from[g + k] << (8 * k);
      return b;
    };
    if (at < depth) {
      const uint64_t b = off ? group(at + off - N) >> (8 * (N - off)) | group(at + off) << (8 * off) : group(at);
      const uint32_t half[2] = {(uint32_t)b, (uint32_t)(b >> 32)};
      union { uint4 vec; T one[N]; } e;
#pragma unroll
      for (int k = 0; k < N; ++k) e.one[k] = Type<T>::put((float)(int8_t)(half[k / 4] >> (8 * (k % 4))) * s);
      if (at >= 0 && at + N <= depth) *reinterpret_cast<uint4*>(to + at) = e.vec;
      else {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (at + k >= 0 && at + k < depth) to[at + k] = e.one[k];
      }
    }
    row += step_rows;
    v += step_at;
    if (v >= per) v -= per, ++row;
  }
}

// ---- the norm's gradient ---------------------------------------------------------------------------------

struct BackArgs {
  const void* h;
  const void* dy;
  const void* dh;
  const void* weight;
  const float* rstd;
  void* dx;
  float* partial;                   // fp32[blocks][depth]
  int64_t rows, h_stride, dy_stride, dh_stride, dx_stride;
  int depth, weight_dtype, warps, groups;   // warps of a row; rows in flight of a block
};

// With xh = h r and g = dy w: dx = r (g - xh mean(g xh)) + dh, dw = sum over the rows of dy xh. A thread keeps its places'
// weights and its sum of dw in registers over all the rows of its group.
template <class T, int MODE, int E, int MOST>
__global__ void __launch_bounds__(MOST) norm_back_kernel(const __grid_constant__ BackArgs a) {
  pdl_begin();
  extern __shared__ float shared[];                // of groups > 1: [groups][depth]
  __shared__ float sums[2][kMostThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool one = a.warps == 1;
  const int tid = one ? lane : threadIdx.x, threads = a.warps * 32, depth = a.depth;
  const int group = one ? warp : 0;
  using M = Mine<T, MODE, E>;
  const M mine{tid, threads, depth, 0};
  float w[E], dw[E];
  mine.load_any(w, a.weight, a.weight_dtype);
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = 0.0f;
  const float inv = 1.0f / (float)depth;
  const T* H = static_cast<const T*>(a.h);
  const T* DY = static_cast<const T*>(a.dy);
  const T* DH = static_cast<const T*>(a.dh);
  // Rows of 16 bits are asked for a row ahead (8192 x 4096 bf16: 58 us, 80 without); in fp32, and entry by entry, that would take the
  // registers of half the rows, and entry by entry even dh comes last (22958 x 693 bf16: 93 us, 117 with all ahead).
  constexpr bool kAhead = sizeof(T) == 2 && MODE != kEntries, kLast = MODE == kEntries;
  typename M::Raw next_h, next_dy, next_dh;
  float next_r = 0.0f;
  auto ahead = [&](int64_t row) {
    mine.fetch(next_h, H + row * a.h_stride);
    mine.fetch(next_dy, DY + row * a.dy_stride);
    if (!kLast && DH) mine.fetch(next_dh, DH + row * a.dh_stride);
    next_r = __ldg(a.rstd + row);
  };
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * a.groups;
  int64_t row = (int64_t)blockIdx.x * a.groups + group;
  if (kAhead && row < a.rows) ahead(row);
  for (; row < a.rows; row += step, turn ^= 1) {
    float h[E], g[E], d[E];
    if (!kAhead) ahead(row);
    M::numbers(h, next_h);
    M::numbers(g, next_dy);
    typename M::Raw dh;
    if (!kLast) dh = next_dh;
    const float r = next_r;
    if (kAhead && row + step < a.rows) ahead(row + step);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      h[i] *= r;
      dw[i] = __fmaf_rn(g[i], h[i], dw[i]);
      g[i] *= w[i];
      s = __fmaf_rn(g[i], h[i], s);
    }
    s = warp_sum(s);
    if (!one) {
      if (lane == 0) sums[turn][warp] = s;
      __syncthreads();                             // the other half is free: all have read it before they came here
      s = warp_sum(lane < a.warps ? sums[turn][lane] : 0.0f);
    }
    s *= inv;
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = r * __fmaf_rn(-h[i], s, g[i]);
    if (DH) {
      if (kLast) mine.fetch(dh, DH + row * a.dh_stride);
      M::numbers(d, dh);
#pragma unroll
      for (int i = 0; i < E; ++i) g[i] += d[i];
    }
    mine.store(static_cast<T*>(a.dx) + row * a.dx_stride, g);
  }
  if (!a.partial) return;
  float* to = a.partial + (int64_t)blockIdx.x * depth;
  if (one) {
#pragma unroll
    for (int j = 0; j < E / M::N; ++j)
#pragma unroll
      for (int i = 0; i < M::N; ++i) {
        const int at = mine.first(j) + i;
        if (at < depth) shared[group * depth + at] = dw[j * M::N + i];
      }
    __syncthreads();
    for (int at = threadIdx.x; at < depth; at += blockDim.x) {
      float s = 0.0f;
      for (int k = 0; k < a.groups; ++k) s += shared[k * depth + at];
      to[at] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < E / M::N; ++j)
#pragma unroll
      for (int i = 0; i < M::N; ++i) {
        const int at = mine.first(j) + i;
        if (at < depth) to[at] = dw[j * M::N + i];
      }
  }
}

// dw = the blocks' sums, in a fixed order: 32 columns a block, 32 parts of the list of blocks each, in four chains (2047 x 1001 fp32: 7.8e-8
// from 64 bits in the 2-norm and 14.4 us, in one chain 1.33e-7 and 16.2; a plain fp32 sum 9.5e-8).
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* partial, int blocks, int depth, float* dweight) {
  pdl_begin();
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = blockIdx.x * 32 + lane;
  float four[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (at < depth) {
    const float* p = partial + at;
    int b = warp;
#pragma unroll 2
    for (; b + 96 < blocks; b += 128)
#pragma unroll
      for (int i = 0; i < 4; ++i) four[i] += __ldg(p + (int64_t)(b + 32 * i) * depth);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (b + 32 * i < blocks) four[i] += __ldg(p + (int64_t)(b + 32 * i) * depth);
  }
  part[warp][lane] = (four[0] + four[1]) + (four[2] + four[3]);
  __syncthreads();
  const float s = warp_sum(part[lane][warp]);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < depth) dweight[col] = s;
}

// ---- launches ---------------------------------------------------------------------------------------------

bool known(int32_t t) { return t == GSPARSE_F32 || t == GSPARSE_BF16 || t == GSPARSE_F16; }
size_t size_of(int32_t t) { return t == GSPARSE_F32 ? 4 : 2; }
bool at_multiple(const void* p, size_t of) { return (reinterpret_cast<uintptr_t>(p) % of) == 0; }

// Whether rows at p, `stride` entries apart, all start at 16-byte boundaries.
bool even(const void* p, int64_t stride, int32_t dtype) {
  return !p || (aligned16(p) && (stride * (int64_t)size_of(dtype)) % 16 == 0);
}

int rows_sizes(int32_t dtype, int64_t rows, int64_t depth, int64_t most = GSPARSE_MAX_NORM_DEPTH) {
  if (!known(dtype) || rows < 0 || depth < 1) return GSPARSE_ERR_INVALID_ARG;
  if (rows > GSPARSE_MAX_ROWS || depth > most) return GSPARSE_ERR_UNSUPPORTED;
  return GSPARSE_OK;
}

// A matrix argument: present, its entries aligned, and where `write`, its rows apart.
bool matrix(const void* p, int64_t stride, int32_t dtype, int64_t rows, int64_t depth, bool write) {
  return p && at_multiple(p, size_of(dtype)) && stride >= (write && rows > 1 ? depth : 0);
}

// Warps of a row and entries a thread: one warp while 16 entries a lane hold the row, then 16 entries a thread; the longest rows
// in 8 bits without a norm, 32 (more in registers with a norm's weights beside them would spill). `more`: places that a shifted row
// takes before its first entry; its warps have 31 lanes.
struct Shape { int warps, entries; };
Shape shape_of(int64_t depth, int more = 0) {
  const int64_t places = depth + more, lanes = more ? 31 : 32;
  if (places <= lanes * 16) return {1, places <= lanes * 8 ? 8 : 16};
  const int e = places <= 32 * lanes * 16 ? 16 : 32;
  return {(int)cdiv(places, lanes * e), e};
}

// Whether rows of 9 to 12 warps are held to the registers of three blocks on an SM (5480 x 5344 bf16: 54 us, 65 with two; 5000 x 5120 fp32,
// which spills then: 71, 68).
template <class T, int MODE, bool NORM>
constexpr bool kThree = NORM && MODE != kEntries && sizeof(T) == 2;

template <class T, int MODE, bool NORM>
void rows_of(const RowArgs& a, const Shape& s, cudaStream_t st) {
  const dim3 grid((unsigned)(s.warps == 1 ? cdiv(a.rows, kRowsPerBlock) : a.rows)), block(s.warps == 1 ? kRowsPerBlock * 32 : s.warps * 32);
  if (s.entries == 8) {
    if constexpr (MODE != kWide) launch(rows_kernel<T, MODE, 8, NORM, 512>, grid, block, 0, st, a);
  } else if (s.entries == 16 && kThree<T, MODE, NORM> && s.warps > 8 && s.warps <= 12)
    launch(rows_kernel<T, MODE, 16, NORM, kThree<T, MODE, NORM> ? 384 : 512>, grid, block, 0, st, a);
  else if (s.entries == 16 && s.warps <= 16) launch(rows_kernel<T, MODE, 16, NORM, 512>, grid, block, 0, st, a);
  else if (s.entries == 16) launch(rows_kernel<T, MODE, 16, NORM, 1024>, grid, block, 0, st, a);
  else if constexpr (!NORM) {
    if (MODE == kWide && s.warps <= 8) launch(rows_kernel<T, MODE, 32, NORM, MODE == kWide ? 256 : 1024>, grid, block, 0, st, a);
    else launch(rows_kernel<T, MODE, 32, NORM, 1024>, grid, block, 0, st, a);
  }
}

template <class T, bool NORM>
void rows_by_mode(const RowArgs& a, const Shape& s, int mode, cudaStream_t st) {
  if (mode == kWide) rows_of<T, kWide, NORM>(a, s, st);
  else if (mode == kVectors) rows_of<T, kVectors, NORM>(a, s, st);
  else if (mode == kShifted) rows_of<T, kShifted, NORM>(a, s, st);
  else rows_of<T, kEntries, NORM>(a, s, st);
}

// The mode of rows whose matrices all start `place` behind a boundary and are `step` apart (modulo 16 bytes), or do not (-1).
struct Places {
  int place = -1, step = -1;
  bool same = true, wide = true;           // wide: at 32-byte boundaries
  void add(const void* p, int64_t stride, int32_t dtype) {
    if (!p) return;
    wide = wide && at_multiple(p, 32) && (stride * (int64_t)size_of(dtype)) % 32 == 0;
    const int a = (int)(reinterpret_cast<uintptr_t>(p) & 15), b = (int)((stride * (int64_t)size_of(dtype)) & 15);
    if (place < 0) place = a, step = b;
    same = same && a == place && b == step;
  }
  bool boundaries() const { return same && place == 0 && step == 0; }
};

template <bool NORM>
int rows_by_type(int32_t dtype, RowArgs& a, const Places& p, cudaStream_t st) {
  const int n = 16 / (int)size_of(dtype);
  const bool vectors = p.boundaries() && a.depth % n == 0 && (!a.weight || aligned16(a.weight));
  Shape s = shape_of(a.depth, vectors || !p.same ? 0 : n - 1);
  // The longest rows of their kernels leave no place for a shift; and with the sum in the place of x or residual a warp's last lane
  // might find the next warp's sum there.
  const bool in_place = a.h && (a.h == a.x || a.h == a.residual);
  const bool wide = vectors && p.wide && s.entries >= 16 && a.depth % (2 * n) == 0 && (!a.weight || at_multiple(a.weight, 32));
  const int mode = wide ? kWide : vectors ? kVectors : p.same && s.warps <= 32 && (!NORM || s.entries <= 16) && !in_place ? kShifted : kEntries;
  if (mode == kEntries) s = shape_of(a.depth);
  // (without a norm half as many threads a row: 8192 x 4096 bf16 34 us with 32 entries a thread, 37 with 16)
  if (!NORM && wide && a.depth >= 1024) s = {(int)cdiv(a.depth, 32 * 32), 32};
  a.warps = s.warps;
  if (dtype == GSPARSE_F32) rows_by_mode<float, NORM>(a, s, mode, st);
  else if (dtype == GSPARSE_BF16) rows_by_mode<__nv_bfloat16, NORM>(a, s, mode, st);
  else rows_by_mode<__half, NORM>(a, s, mode, st);
  return launch_status();
}

template <class T, int MODE>
void back_of(const BackArgs& a, const Shape& s, int blocks, size_t smem, cudaStream_t st) {
  const dim3 grid((unsigned)blocks), block((unsigned)(a.groups * s.warps * 32));
  if (s.entries == 8) launch(norm_back_kernel<T, MODE, 8, 512>, grid, block, smem, st, a);
  else if (s.warps <= 16) launch(norm_back_kernel<T, MODE, 16, 512>, grid, block, smem, st, a);
  else launch(norm_back_kernel<T, MODE, 16, 1024>, grid, block, smem, st, a);
}

template <class T>
void back_by_mode(const BackArgs& a, const Shape& s, bool vec, bool pairs, int blocks, size_t smem, cudaStream_t st) {
  if (vec) back_of<T, kVectors>(a, s, blocks, smem, st);
  else if (sizeof(T) == 2 && pairs) back_of<T, sizeof(T) == 2 ? kWords : kEntries>(a, s, blocks, smem, st);
  else back_of<T, kEntries>(a, s, blocks, smem, st);
}

int back_groups(const Shape& s) { return s.warps == 1 ? 8 : 1; }

// Rows that a group takes at least: 4000 x 512 bf16 12.4, 9.6 and 10.2 us with 1, 2 and 4 (fewer parts to join, fewer rows at a time).
constexpr int kBackRows = 2;

// Blocks of the gradient: what the SMs hold at once (about 1024 threads each), at most one a group of rows.
int back_blocks(int64_t rows, const Shape& s) {
  const int groups = back_groups(s), threads = groups * s.warps * 32;
  const int64_t most = sm_count() * (int64_t)(threads >= 1024 ? 1 : 1024 / threads);
  const int64_t need = cdiv(rows, (int64_t)groups * kBackRows);
  return (int)(need < most ? need : most);
}

template <class T>
void dequant_of(const int8_t* q, int64_t q_stride, const float* scale, int64_t rows, int depth, void* out, int64_t out_stride, cudaStream_t st) {
  constexpr int N = Type<T>::N;
  const bool even = aligned16(out) && (rows == 1 || (out_stride * (int64_t)sizeof(T)) % 16 == 0);
  const int per = even ? (int)cdiv(depth, 16) : (int)cdiv(depth + N - 1, N);
  const int64_t blocks = cdiv(rows * per, 256), most = (int64_t)sm_count() * (even ? 32 : 64);
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if (even) launch(dequant_kernel<T>, grid, dim3(256), 0, st, q, q_stride, scale, rows, depth, static_cast<T*>(out), out_stride);
  else launch(dequant_shifted_kernel<T>, grid, dim3(256), 0, st, q, q_stride, scale, rows, depth, static_cast<T*>(out), out_stride, per);
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" {

int gsparse_quantize_rows(const void* x, int32_t dtype, int64_t rows, int64_t depth, int64_t row_stride, int8_t* q, int64_t q_stride,
                          float* scale, gsparse_stream stream) {
  const int st = rows_sizes(dtype, rows, depth, GSPARSE_MAX_DEPTH);
  if (st != GSPARSE_OK || rows == 0) return st;
  if (!matrix(x, row_stride, dtype, rows, depth, false)) return GSPARSE_ERR_INVALID_ARG;
  if (!q || !scale || !aligned16(q) || q_stride % 16 || q_stride < depth || !at_multiple(scale, 4)) return GSPARSE_ERR_INVALID_ARG;
  RowArgs a{};
  a.x = x;
  a.x_stride = row_stride;
  a.q = q;
  a.q_stride = q_stride;
  a.scale = scale;
  a.rows = rows;
  a.depth = (int)depth;
  Places p;
  p.add(x, row_stride, dtype);
  return rows_by_type<false>(dtype, a, p, (cudaStream_t)stream);
}

int gsparse_dequantize_rows(const int8_t* q, int64_t q_stride, const float* scale, int64_t rows, int64_t depth, void* out, int32_t dtype,
                            int64_t out_stride, gsparse_stream stream) {
  const int st = rows_sizes(dtype, rows, depth, GSPARSE_MAX_DEPTH);
  if (st != GSPARSE_OK || rows == 0) return st;
  if (!q || !scale || !aligned16(q) || q_stride % 16 || q_stride < depth || !at_multiple(scale, 4)) return GSPARSE_ERR_INVALID_ARG;
  if (!matrix(out, out_stride, dtype, rows, depth, true)) return GSPARSE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == GSPARSE_F32) dequant_of<float>(q, q_stride, scale, rows, (int)depth, out, out_stride, s);
  else if (dtype == GSPARSE_BF16) dequant_of<__nv_bfloat16>(q, q_stride, scale, rows, (int)depth, out, out_stride, s);
  else dequant_of<__half>(q, q_stride, scale, rows, (int)depth, out, out_stride, s);
  return launch_status();
}

int gsparse_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const void* weight,
                     int32_t weight_dtype, int32_t dtype, int64_t rows, int64_t depth, float eps, void* h, int64_t h_stride, void* y,
                     int64_t y_stride, int8_t* q, int64_t q_stride, float* scale, float* rstd, gsparse_stream stream) {
  const int st = rows_sizes(dtype, rows, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(weight_dtype) || !(eps >= 0x1p-126f) || !isfinite(eps)) return GSPARSE_ERR_INVALID_ARG;
  if (rows == 0) return GSPARSE_OK;
  if (!matrix(x, x_stride, dtype, rows, depth, false) || !weight || !at_multiple(weight, size_of(weight_dtype)))
    return GSPARSE_ERR_INVALID_ARG;
  if (residual && !matrix(residual, residual_stride, dtype, rows, depth, false)) return GSPARSE_ERR_INVALID_ARG;
  if (h && !matrix(h, h_stride, dtype, rows, depth, true)) return GSPARSE_ERR_INVALID_ARG;
  if (y && !matrix(y, y_stride, dtype, rows, depth, true)) return GSPARSE_ERR_INVALID_ARG;
  if ((h && h == x && h_stride != x_stride) || (h && h == residual && h_stride != residual_stride)) return GSPARSE_ERR_INVALID_ARG;
  if ((q != nullptr) != (scale != nullptr)) return GSPARSE_ERR_INVALID_ARG;
  if (q && (!aligned16(q) || q_stride % 16 || q_stride < depth || !at_multiple(scale, 4))) return GSPARSE_ERR_INVALID_ARG;
  if (!at_multiple(rstd, 4)) return GSPARSE_ERR_INVALID_ARG;
  RowArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h = h;
  a.y = y;
  a.q = q;
  a.scale = scale;
  a.rstd = rstd;
  a.rows = rows;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.h_stride = h_stride;
  a.y_stride = y_stride;
  a.q_stride = q_stride;
  a.depth = (int)depth;
  a.weight_dtype = weight_dtype;
  a.eps = eps;
  a.inv_depth = 1.0 / (double)depth;
  Places p;
  p.add(x, x_stride, dtype);
  p.add(residual, residual_stride, dtype);
  p.add(h, h_stride, dtype);
  p.add(y, y_stride, dtype);
  return rows_by_type<true>(dtype, a, p, (cudaStream_t)stream);
}

size_t gsparse_rms_norm_backward_workspace_size(int64_t rows, int64_t depth) {
  if (rows_sizes(GSPARSE_F32, rows, depth) != GSPARSE_OK) return 0;
  return 256 + (size_t)back_blocks(rows, shape_of(depth)) * (size_t)depth * sizeof(float);
}

int gsparse_rms_norm_backward(const void* h, int64_t h_stride, const void* weight, int32_t weight_dtype, const float* rstd,
                              const void* dy, int64_t dy_stride, const void* dh, int64_t dh_stride, int32_t dtype, int64_t rows,
                              int64_t depth, void* dx, int64_t dx_stride, float* dweight, void* workspace, size_t workspace_bytes,
                              gsparse_stream stream) {
  const int st = rows_sizes(dtype, rows, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(weight_dtype) || !at_multiple(dweight, 4)) return GSPARSE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)depth * sizeof(float), s) != cudaSuccess) {
      cudaGetLastError();
      return GSPARSE_ERR_CUDA;
    }
    return GSPARSE_OK;
  }
  if (!weight || !at_multiple(weight, size_of(weight_dtype)) || !rstd || !at_multiple(rstd, 4)) return GSPARSE_ERR_INVALID_ARG;
  if (!matrix(h, h_stride, dtype, rows, depth, false) || !matrix(dy, dy_stride, dtype, rows, depth, false) ||
      !matrix(dx, dx_stride, dtype, rows, depth, true))
    return GSPARSE_ERR_INVALID_ARG;
  if (dh && !matrix(dh, dh_stride, dtype, rows, depth, false)) return GSPARSE_ERR_INVALID_ARG;
  if ((dx == h && dx_stride != h_stride) || (dx == dy && dx_stride != dy_stride) || (dx == dh && dx_stride != dh_stride))
    return GSPARSE_ERR_INVALID_ARG;
  const Shape shape = shape_of(depth);
  const int blocks = back_blocks(rows, shape);
  Carver c(workspace);
  float* partial = c.take<float>((int64_t)blocks * depth);
  if (dweight && (!workspace || !at_multiple(workspace, 256) || workspace_bytes < c.off)) return GSPARSE_ERR_WORKSPACE;
  BackArgs a{};
  a.h = h;
  a.dy = dy;
  a.dh = dh;
  a.weight = weight;
  a.rstd = rstd;
  a.dx = dx;
  a.partial = dweight ? partial : nullptr;
  a.rows = rows;
  a.h_stride = h_stride;
  a.dy_stride = dy_stride;
  a.dh_stride = dh_stride;
  a.dx_stride = dx_stride;
  a.depth = (int)depth;
  a.weight_dtype = weight_dtype;
  a.warps = shape.warps;
  a.groups = back_groups(shape);
  const bool vec = depth % (16 / (int64_t)size_of(dtype)) == 0 && aligned16(weight) && even(h, h_stride, dtype) &&
                   even(dy, dy_stride, dtype) && even(dh, dh_stride, dtype) && even(dx, dx_stride, dtype);
  const size_t smem = shape.warps == 1 ? (size_t)a.groups * (size_t)depth * sizeof(float) : 0;   // at most 16 KB
  auto words = [&](const void* p, int64_t stride) { return !p || (at_multiple(p, 4) && stride % 2 == 0); };
  const bool pairs = size_of(dtype) == 2 && depth % 2 == 0 && words(h, h_stride) && words(dy, dy_stride) && words(dh, dh_stride) && words(dx, dx_stride);
  if (dtype == GSPARSE_F32) back_by_mode<float>(a, shape, vec, false, blocks, smem, s);
  else if (dtype == GSPARSE_BF16) back_by_mode<__nv_bfloat16>(a, shape, vec, pairs, blocks, smem, s);
  else back_by_mode<__half>(a, shape, vec, pairs, blocks, smem, s);
  if (dweight) launch(norm_join_kernel, dim3((unsigned)cdiv(depth, 32)), dim3(1024), 0, s, (const float*)partial, blocks, (int)depth, dweight);
  return launch_status();
}

}  // extern "C"

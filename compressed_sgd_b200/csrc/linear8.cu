// The product of rows in 8 bits, and its gradients, on the fifth-generation tensor cores.
//
// One kernel serves all three: D[m][n] = sum over s of A(m, s) B(n, s), with pairs of CTAs that take 256 x 256 tiles of D.
//   product      A = x [tokens][depth], B = w [channels][depth], both int8 and s along their rows; D in 32-bit integers.
//   grad_input   A = dout [tokens][channels], s along its rows; B = w's values in bf16 [channels][depth], s across its rows.
//   grad_weight  A = dout [tokens][channels] and B = x's values in bf16 [tokens][depth], s across the rows of both.
// The values of rows in 8 bits are bf16 numbers (rows8.cu), so the gradients' products are exact in fp32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tiles.cuh"

namespace gs {
namespace {

constexpr int kRowBytes = 128;             // of an operand's row in a stage: 128 int8 or 64 bf16 (one swizzle atom)
constexpr int kOperand = 128 * kRowBytes;  // bytes of one operand of one CTA in a stage
constexpr int kBox = 32 * 128;             // a warp's part of the result on its way out: 32 rows of 128 bytes

constexpr int kSide = 128;                 // columns of a warp that takes results out: eight of them take a CTA's part of a tile

// Few rows that every pair reads at about the same time are slow to come by (16 tokens against 32000 x 4096 weights: 100 us, 64
// tokens: 31): they are copied, and the pairs read different copies.
// The copies take about half a megabyte (8 tokens of 512 in 16 copies, 64 KB: 40 us; in 74: 17).
constexpr int64_t kCopyBytes = 96 << 10, kCopiesBytes = 512 << 10;

// Integers leave the tensor memory once a tile, but soon (a depth of 512 takes a pair a microsecond): two groups of eight warps, which
// take the tiles in turn. Sums in bf16 stay in registers over a tile: one group, with the registers that the other warps give up.
template <bool INT> struct Layout {
  static constexpr int warps = INT ? 16 : 8;                   // that take results out
  static constexpr int threads = (warps + (INT ? 2 : 4)) * 32; // setmaxnreg goes by groups of four warps
  static constexpr int stages = INT ? 5 : 6;
  static constexpr int stage_bytes = 2 * kOperand;
  static constexpr int box_at = stages * stage_bytes;
  static constexpr int scale_at = box_at + warps * kBox;
  static constexpr int bar_at = scale_at + (INT ? 2 * kTile * 4 : 0);
  static constexpr int shared = bar_at + 256;
};
using LB = Layout<false>;
constexpr int kMore = 216, kFewer = 72;      // registers of these and of the others, out of the 168 of the launch
static_assert(LB::warps * 32 * kMore + 128 * kFewer <= LB::threads * 168, "");

struct TileArgs {
  CUtensorMap a, b, out, part;
  const float* row_scale;                  // of the integer product
  const float* col_scale;
  void* result;
  int64_t result_stride;
  int64_t as_tiles;                        // columns of D that the tensor map describes: a copy ends at a multiple of 16 bytes
  int32_t* d_status;
  int64_t rows, cols;                      // of D
  Order order;
  int blocks, plane_blocks;                // of 128 bytes along s, all planes; of one plane
  int chunk;                               // blocks of bf16 that are summed in the tensor core
  int pairs, waves;                        // tiles below waves * pairs are whole; the others are split
  int piece, group, span;                  // blocks of a pair's part of the split tiles (0: none are split), and of a tile's parts; see Plan
  int stacked;                             // the planes are rows of A: every tile is a part
  int copies;                              // of the integer A, one after another
  int keep_a, keep_b;                      // how long the second-level cache should keep the operands' lines
  int out_dtype;
};

// ---- instructions ----------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Waits for a phase; false after about a second. What these barriers guard is copied and multiplied by asynchronous units and read
// from tensor memory, so neither the waits nor the arrivals order plain memory accesses over the cluster: a release of that
// scope before each arrival was a third of the warps' time that take results out. The time that a wait may sleep (in ns) keeps the
// warps that wait from the issue slots and from the power that the others need: 282 against 268 us for the gradient by 85000 x 512
// weights over 4000 tokens.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  uint32_t ok = 0;
  const long long t0 = clock64();
  do {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(at), "r"(parity) : "memory");
  } while (!ok && clock64() - t0 < kWaitCycles);
  return ok != 0;
}

__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Copies of a box into this CTA's shared memory that count on a barrier of the pair's first CTA.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t keep) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], "
      "[%4], %5;" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar), "l"(keep)
      : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar, uint64_t keep) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4}], [%5], %6;" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(keep)
      : "memory");
}

// Policies of the second-level cache: lines of an operand that is read again and again, of one that passes once, and of others.
__device__ __forceinline__ uint64_t policy(int keep) {
  uint64_t p;
  if (keep > 0) asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  else if (keep < 0) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// A tile in shared memory, swizzled by 128 bytes. Rows along s (a row of 128 bytes per m): groups of 8 rows 1024 bytes apart.
// Rows across s (a row of 64 m per s): groups of 8 s 1024 bytes apart, the next 64 m 8192 bytes on.
__device__ __forceinline__ uint64_t tile_of(uint32_t addr, bool across) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)(across ? 8192 >> 4 : 1) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

template <bool INT>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add) {
  if constexpr (INT)
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b),
                 "r"(what), "r"((uint32_t)add)
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b),
                 "r"(what), "r"((uint32_t)add)
                 : "memory");
}

// The barrier at this place in both CTAs, once what was issued before has been done.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}

__device__ __forceinline__ void load_columns(uint32_t (&v)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]),
        "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
        "=r"(v[31])
      : "r"(at));
}
__device__ __forceinline__ void columns_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- the way out --------------------------------------------------------------------------------------------

template <class T> struct Pack;
template <> struct Pack<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint4 of(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <> struct Pack<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&p);
  }
  static __device__ __forceinline__ uint4 of(const float* v) { return make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7])); }
};
template <> struct Pack<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&p);
  }
  static __device__ __forceinline__ uint4 of(const float* v) { return make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7])); }
};

// 32 of a row's results (lane = row) into the warp's box, from the 16-byte place `at` on. Rows are swizzled as the tensor maps say,
// which also spreads the lanes over the banks.
template <class T>
__device__ __forceinline__ void into_box(char* box, int lane, int at, const float* v) {
#pragma unroll
  for (int j = 0; j < 32 / Pack<T>::N; ++j)
    *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(box + lane * 128 + ((lane & 7) << 4)) ^ (uintptr_t)((at + j) << 4)) = Pack<T>::of(v + j * Pack<T>::N);
}

// A box of 32 rows that no tensor map describes: row by row, 128 bytes of entries side by side.
template <class T>
__device__ void box_to_rows(const char* box, int lane, T* out, int64_t stride, int64_t row, int64_t col, int64_t rows, int64_t cols) {
  constexpr int N = 4 / (int)sizeof(T);
  const int n = (int)min((int64_t)32, rows - row);
  const int64_t mine = col + lane * N;
  const int have = (int)max((int64_t)0, min((int64_t)N, cols - mine));
  T* to = out + row * stride + mine;
  const char* from = box + (lane & 3) * 4;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 8) {             // eight rows under way at a time
    uint32_t raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = *reinterpret_cast<const uint32_t*>(from + (r0 + i) * 128 + (((lane >> 2) ^ i) << 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T* e = reinterpret_cast<const T*>(&raw[i]);
      if (r0 + i < n) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (k < have) to[k] = e[k];
      }
      to += stride;
    }
  }
}

// Two sums times their row's scale, then times their columns' scales, each rounded (two numbers an instruction).
__device__ __forceinline__ void scaled(float& u, float& v, uint32_t a, uint32_t b, float row, float x, float y) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %4};\n mov.b64 r, {%5, %6};\n mul.rn.f32x2 p, p, q;\n"
      " mul.rn.f32x2 p, p, r;\n mov.b64 {%0, %1}, p;\n}"
      : "=f"(u), "=f"(v)
      : "f"(__int2float_rn((int)a)), "f"(__int2float_rn((int)b)), "f"(row), "f"(x), "f"(y));
}

// A warp's box on its way.
struct Way {
  char* box;
  int lane;

  // Once what it held has been read.
  __device__ __forceinline__ void next() {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }
  __device__ __forceinline__ void send(const CUtensorMap* map, int64_t x, int64_t y) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) store_box(map, (int)x, (int)y, smem_u32(box));
  }
};

// A warp's 32 x 32 results v at (row, col) of D, the `half`-th of a box of 16-bit types.
template <class T>
__device__ __forceinline__ void put_result(const TileArgs& a, Way& way, int half, const float* v, int64_t row, int64_t col) {
  constexpr bool narrow = sizeof(T) == 2;
  if (!narrow || half == 0) way.next();
  into_box<T>(way.box, way.lane, narrow ? half * 4 : 0, v);
  if (narrow && half == 0) return;
  const int64_t x = narrow ? col - 32 : col;
  if (row >= a.rows || x >= a.cols) return;
  if (x + 128 / (int)sizeof(T) <= a.as_tiles || a.as_tiles == a.cols) {
    way.send(&a.out, x, row);
  } else {
    __syncwarp();
    box_to_rows<T>(way.box, way.lane, static_cast<T*>(a.result), a.result_stride, row, x, a.rows, a.cols);
    __syncwarp();
  }
}

__device__ __forceinline__ void put(const TileArgs& a, Way& way, int half, const float* v, int64_t row, int64_t col) {
  if (a.out_dtype == GSPARSE_F32) put_result<float>(a, way, half, v, row, col);
  else if (a.out_dtype == GSPARSE_BF16) put_result<__nv_bfloat16>(a, way, half, v, row, col);
  else put_result<__half>(a, way, half, v, row, col);
}

// A part of a tile's sums, as they are: row r of slot k at row k * 256 + r of the workspace. What lies outside D is left out.
__device__ __forceinline__ void put_part(const TileArgs& a, Way& way, const float* v, int64_t row, int col, bool inside) {
  if (!inside) return;
  way.next();
  into_box<float>(way.box, way.lane, 0, v);
  way.send(&a.part, col, row);
}

// ---- the kernel -----------------------------------------------------------------------------------------------

// The first warps take results out (warp w the lanes 32 (w % 4) and the columns 128 (w / 4 % 2) on), the next loads, one more
// multiplies (of the pair's first CTA, for both). The loads run ahead over all of a pair's parts; the tensor memory holds two tiles of sums.
//
// The sums in bf16 are taken out of the tensor core every `chunk` blocks of 64 and added up in fp32 registers, since its
// accumulation cuts off, towards zero.
template <bool INT, bool A_ACROSS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<INT>::threads, 1) tile_kernel(const __grid_constant__ TileArgs a) {
  extern __shared__ __align__(1024) char smem[];
  using L = Layout<INT>;
  constexpr bool kAcross = !INT;                               // B's rows
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar_at);
  uint64_t* empty = full + L::stages;
  uint64_t* sums_full = empty + L::stages;
  uint64_t* sums_empty = sums_full + 2;
  uint64_t* drained = sums_empty + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sums_full + i, 1);
      mbar_init(sums_empty + i, 2 * 8);
    }
    mbar_init(drained, 1);
    fence_mbarrier_init();
  }
  if (warp == L::warps + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    fence_before();
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_begin();

  bool ok = true;
  Part p;
  if (warp >= L::warps) {
    if constexpr (!INT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewer));
    if (warp == L::warps && lane == 0) {
      uint32_t n = 0, s = 0, turn = 0;                         // stages filled so far; the next, and its turn
      const uint64_t keep_a = policy(a.keep_a), keep_b = policy(a.keep_b);
      const int copy = INT ? pair % a.copies : 0;
      for (int i = 0; ok && part_of(a, pair, i, p); ++i) {
        const int m = p.m * kTile + (int)rank * 128, c = p.n * kTile + (int)rank * 128;
        int plane = p.from / a.plane_blocks, k = p.from - plane * a.plane_blocks;
        for (int kb = p.from; kb < p.to; ++kb, ++n) {
          if (turn && !(ok = wait_phase(empty + s, (turn - 1) & 1))) break;
          if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * L::stage_bytes);
          const uint32_t bar = in_cta(smem_u32(full + s), 0);
          const uint32_t at = smem_u32(smem + s * L::stage_bytes);
          if constexpr (INT) {
            load_box(at, &a.a, k * 128, m, copy, bar, keep_a);
            load_box(at + kOperand, &a.b, k * 128, c, bar, keep_b);
          } else {
            if constexpr (A_ACROSS) {
              load_box(at, &a.a, m, k * 64, plane, bar, keep_a);
              load_box(at + kOperand / 2, &a.a, m + 64, k * 64, plane, bar, keep_a);
            } else {
              load_box(at, &a.a, k * 64, m, plane, bar, keep_a);
            }
            load_box(at + kOperand, &a.b, c, k * 64, bar, keep_b);
            load_box(at + kOperand + kOperand / 2, &a.b, c + 64, k * 64, bar, keep_b);
          }
          if (++s == L::stages) s = 0, ++turn;
          if (++k == a.plane_blocks) k = 0, ++plane;
        }
      }
      if (!ok) {
        raise(a.d_status, GSPARSE_DERR_TIMEOUT);
        if (rank == 0)                                         // the copies under way, of both CTAs
          for (uint32_t b = n > L::stages ? n - L::stages : 0; b < n; ++b) wait_phase(full + b % L::stages, (b / L::stages) & 1);
      }
    }
    if (warp == L::warps + 1 && lane == 0 && rank == 0) {
      constexpr uint32_t what = (INT ? 2u << 4 : 1u << 4) | 1u << 7 | 1u << 10 | (A_ACROSS ? 1u << 15 : 0u) | (kAcross ? 1u << 16 : 0u) |
                                (uint32_t)(kTile >> 3) << 17 | (uint32_t)(kTile >> 4) << 24;
      uint32_t s = 0, turn = 0, c = 0;                         // the next stage and its turn, sums begun
      for (int i = 0; ok && part_of(a, pair, i, p); ++i) {
        for (int kb = p.from; ok && kb < p.to; ++c) {
          const int end = INT ? p.to : min(p.to, kb + a.chunk);
          const uint32_t buf = c & 1, d = tmem + buf * kTile;
          if (c >= 2 && !(ok = wait_phase(sums_empty + buf, (c / 2 - 1) & 1))) break;
          fence_after();
          for (bool add = false; kb < end; ++kb) {
            if (!(ok = wait_phase(full + s, turn & 1))) break;
            fence_after();
            const uint32_t at = smem_u32(smem + s * L::stage_bytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {                      // 32 bytes along s, or 16 rows across it
              multiply<INT>(d, tile_of(at + k * (A_ACROSS ? 2048 : 32), A_ACROSS), tile_of(at + kOperand + k * (kAcross ? 2048 : 32), kAcross), what,
                            add);
              add = true;
            }
            commit(empty + s);
            if (++s == L::stages) s = 0, ++turn;
          }
          if (ok) commit(sums_full + buf);
        }
      }
      if (!ok) {
        raise(a.d_status, GSPARSE_DERR_TIMEOUT);
        commit(drained);
        wait_phase(drained, 0);
      }
    }
  } else {
    if constexpr (!INT) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMore));
    const int quarter = warp & 3, side = (warp >> 2) & 1, group = warp >> 3;
    const int first_row = (int)rank * 128 + quarter * 32, first_col = side * kSide;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + first_col;
    const uint32_t give = in_cta(smem_u32(sums_empty), 0);
    Way way{smem + L::box_at + warp * kBox, lane};
    if constexpr (INT) {
      // Two groups of eight warps take the parts in turn, so that one converts while the other waits, loads or sends. The scales of
      // a part's rows, and of its columns for the four warps that take the same ones, are read a part ahead.
      float row_scale = 0.0f, col_scale = 0.0f;
      const int mine_of = quarter * 32 + lane;
      auto scales_of = [&](const Part& q) {
        const int64_t row = (int64_t)q.m * kTile + first_row + lane, col = (int64_t)q.n * kTile + first_col + mine_of;
        row_scale = row < a.rows ? __ldg(a.row_scale + row) : 0.0f;
        col_scale = col < a.cols ? __ldg(a.col_scale + col) : 0.0f;
      };
      int i = group;
      bool more = part_of(a, pair, i, p);
      if (more) scales_of(p);
      for (uint32_t turn = 0; more; ++turn) {      // (after a wait that gave up: on to the end, since four warps meet at a barrier)
        float* scales = reinterpret_cast<float*>(smem + L::scale_at) + group * kTile + first_col;
        asm volatile("bar.sync %0, 128;" ::"r"(warp / 4 + 1) : "memory");      // the last part's scales have been used
        scales[mine_of] = col_scale;
        const float mine = row_scale;
        const int64_t row = (int64_t)p.m * kTile + first_row, col = (int64_t)p.n * kTile + first_col;
        const int64_t part_row = (int64_t)p.slot * kTile + first_row;
        const bool whole = p.whole;
        more = part_of(a, pair, i += 2, p);
        if (more) scales_of(p);
        asm volatile("bar.sync %0, 128;" ::"r"(warp / 4 + 1) : "memory");
        if (!(ok = ok && wait_phase(sums_full + group, turn & 1))) continue;
        fence_after();
#pragma unroll
        for (int j = 0; j < kSide / 32; ++j) {
          uint32_t raw[32];
          load_columns(raw, lanes + group * kTile + j * 32);
          columns_loaded();
          if (j == kSide / 32 - 1) {
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(give + group * 8);
          }
          float v[32];
          if (whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 f = *reinterpret_cast<const float4*>(scales + j * 32 + k);
              scaled(v[k], v[k + 1], raw[k], raw[k + 1], mine, f.x, f.y);
              scaled(v[k + 2], v[k + 3], raw[k + 2], raw[k + 3], mine, f.z, f.w);
            }
            put(a, way, j & 1, v, row, col + j * 32);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(raw[k]);
            put_part(a, way, v, part_row, first_col + j * 32, row < a.rows && col + j * 32 < a.cols);
          }
        }
      }
    } else {
      uint32_t c = 0;
      for (int i = 0; part_of(a, pair, i, p); ++i) {
        float sum[kSide];
        for (int kb = p.from; ok && kb < p.to; kb += a.chunk, ++c) {
          const uint32_t buf = c & 1;
          if (!(ok = wait_phase(sums_full + buf, (c / 2) & 1))) break;
          fence_after();
#pragma unroll
          for (int j = 0; j < kSide; j += 32) {
            uint32_t raw[32];
            load_columns(raw, lanes + buf * kTile + j);
            columns_loaded();
            if (kb == p.from) {
#pragma unroll
              for (int k = 0; k < 32; ++k) sum[j + k] = __uint_as_float(raw[k]);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) sum[j + k] += __uint_as_float(raw[k]);
            }
          }
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(give + buf * 8);
        }
        if (!ok) break;
        const int64_t row = (int64_t)p.m * kTile + first_row, col = (int64_t)p.n * kTile + first_col;
        const int64_t part_row = (int64_t)p.slot * kTile + first_row;
#pragma unroll
        for (int j = 0; j < kSide / 32; ++j) {
          if (p.whole) put(a, way, j & 1, sum + j * 32, row, col + j * 32);
          else put_part(a, way, sum + j * 32, part_row, first_col + j * 32, row < a.rows && col + j * 32 < a.cols);
        }
      }
    }
    if (!ok && lane == 0) raise(a.d_status, GSPARSE_DERR_TIMEOUT);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  // nobody leaves while the other CTA may still reach into its shared or tensor memory
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == L::warps + 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---- split tiles -------------------------------------------------------------------------------------------------

struct JoinArgs {
  const float* part;
  const float* row_scale;
  const float* col_scale;
  void* out;
  int64_t out_stride, rows, cols;
  Order order;
  int first_tile, blocks, piece, group, span;
  int planes, plane_rows;                  // of stacked planes: rows r, plane_rows + r, ... are added up
};

// The parts of a split tile added up, along s: WARPS warps take a row of it, parts warp, warp + WARPS, ... each, 8 entries a lane.
template <bool INT, class T, int WARPS>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
  pdl_begin();
  __shared__ uint32_t joined[WARPS > 1 ? WARPS : 1][WARPS > 1 ? kTile : 1];
  constexpr int kRows = 8 / WARPS, kBlocks = kTile / kRows;    // rows of a block, blocks of a tile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x / kBlocks, tile = a.first_tile + t;
  const int r = (blockIdx.x % kBlocks) * kRows + warp / WARPS, c = lane * 8;
  const Parts parts = parts_of(t, a.blocks, a.piece, a.group, a.span);
  if (parts.count == 1 && a.planes == 1) return;   // whole after all
  const int all = parts.count * a.planes;
  int m, n;
  place_of(tile, a.order, m, n);
  const int64_t row = (int64_t)m * kTile + r, col = (int64_t)n * kTile + c;
  if (row >= a.rows || (WARPS == 1 && col >= a.cols)) return;  // (with more warps they all do, or none)
  uint32_t sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};     // -0 + 0 is 0: as good as the first part itself
  for (int at = warp % WARPS; at < all && col < a.cols; at += 4 * WARPS) {   // four parts under way at a time
    uint4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at + i * WARPS >= all) break;
      const int plane = (at + i * WARPS) / parts.count;
      const int64_t slot = parts.slot(at + i * WARPS - plane * parts.count);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.part) + (slot * kTile + plane * a.plane_rows + r) * kTile + c;
      x[i] = __ldg(reinterpret_cast<const uint4*>(p));
      y[i] = __ldg(reinterpret_cast<const uint4*>(p + 4));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at + i * WARPS >= all) break;
      const uint32_t v[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (INT) sum[k] += v[k];
        else sum[k] = __float_as_uint(__uint_as_float(sum[k]) + __uint_as_float(v[k]));
      }
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) joined[warp][k * 32 + lane] = sum[k];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t v = joined[w][k * 32 + lane];
        if constexpr (INT) sum[k] += v;
        else sum[k] = __float_as_uint(__uint_as_float(sum[k]) + __uint_as_float(v));
      }
  }
  if (col >= a.cols) return;
  T* out = static_cast<T*>(a.out) + row * a.out_stride + col;
  const float mine = INT ? __ldg(a.row_scale + row) : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (col + i >= a.cols) break;
    float v;
    if constexpr (INT) v = __int2float_rn((int)sum[i]) * mine * __ldg(a.col_scale + col + i);
    else v = __uint_as_float(sum[i]);
    if constexpr (sizeof(T) == 4) out[i] = v;
    else if constexpr (__is_same(T, __nv_bfloat16)) out[i] = __float2bfloat16_rn(v);
    else out[i] = __float2half_rn(v);
  }
}

// ---- few tokens ----------------------------------------------------------------------------------------------------

struct FewArgs {
  const int8_t* x;
  const int8_t* w;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t x_stride, w_stride, out_stride, channels;
  int tokens, depth, out_dtype;
};

// The last bytes of a row in 8 bits, from `at` on, and zeros: what stands behind the row is not read.
__device__ __noinline__ uint4 last_bytes(const int8_t* row, int at, int depth) {
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + i < depth) v[i / 4] |= (uint32_t)(uint8_t)row[at + i] << (8 * (i % 4));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// ROWS channels of the weights pass once, 16 bytes a lane, against the tokens' rows (by way of the first-level cache): the call is
// the weights' way from memory. With SPLIT the eight warps of a block share its channels along the depth, else each has its own.
template <int TOKENS, int ROWS, bool SPLIT>
__global__ void __launch_bounds__(256) few_kernel(const __grid_constant__ FewArgs a) {
  pdl_begin();
  __shared__ int parts[SPLIT ? 8 : 1][TOKENS][ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = (SPLIT ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + warp) * ROWS;
  if (first >= a.channels) return;                 // (with SPLIT the whole block)
  const int8_t* x = a.x;
  const int8_t* w = a.w + first * a.w_stride;
  const int last_row = (int)min((int64_t)ROWS - 1, a.channels - 1 - first), last_token = a.tokens - 1;
  int sum[ROWS][TOKENS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) sum[r][t] = 0;
  for (int at = (SPLIT ? threadIdx.x : lane) * 16; at < a.depth; at += SPLIT ? 4096 : 512) {
    uint4 wr[ROWS], xt[TOKENS];
    const bool all = at + 16 <= a.depth;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int8_t* p = w + min(r, last_row) * a.w_stride;
      wr[r] = all ? __ldg(reinterpret_cast<const uint4*>(p + at)) : last_bytes(p, at, a.depth);
    }
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      const int8_t* p = x + min(t, last_token) * a.x_stride;
      xt[t] = all ? __ldg(reinterpret_cast<const uint4*>(p + at)) : last_bytes(p, at, a.depth);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int t = 0; t < TOKENS; ++t) {
        int s = __dp4a((int)wr[r].x, (int)xt[t].x, sum[r][t]);
        s = __dp4a((int)wr[r].y, (int)xt[t].y, s);
        s = __dp4a((int)wr[r].z, (int)xt[t].z, s);
        sum[r][t] = __dp4a((int)wr[r].w, (int)xt[t].w, s);
      }
  }
  // result (t, r) to lane t * ROWS + r (of the whole block with SPLIT)
  constexpr int N = TOKENS * ROWS;
  static_assert(N <= 32, "");
  int mine = 0;
#pragma unroll
  for (int t = 0; t < TOKENS; ++t)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int s = __reduce_add_sync(kFull, sum[r][t]);
      if (lane == t * ROWS + r) mine = s;
    }
  const int t = lane / ROWS, r = lane % ROWS;
  if constexpr (SPLIT) {
    if (lane < N) parts[warp][t][r] = mine;
    __syncthreads();
    if (warp != 0) return;
    if (lane < N) {
      mine = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) mine += parts[k][t][r];
    }
  }
  if (lane >= N || t > last_token || r > last_row) return;
  const float v = __int2float_rn(mine) * __ldg(a.x_scale + t) * __ldg(a.w_scale + first + r);
  const int64_t to = t * a.out_stride + first + r;
  if (a.out_dtype == GSPARSE_F32) static_cast<float*>(a.out)[to] = v;
  else if (a.out_dtype == GSPARSE_BF16) static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(v);
  else static_cast<__half*>(a.out)[to] = __float2half_rn(v);
}

// Copies of rows in 8 bits, one after another; a block takes a row of one of them.
__global__ void __launch_bounds__(128) copies_kernel(const int8_t* x, int64_t x_stride, int tokens, int depth, int8_t* out, int64_t out_stride) {
  pdl_begin();
  const int copy = blockIdx.x / tokens, t = blockIdx.x - copy * tokens;
  const int8_t* row = x + t * x_stride;
  int8_t* to = out + ((int64_t)copy * tokens + t) * out_stride;
  for (int at = threadIdx.x * 16; at < depth; at += 128 * 16)
    *reinterpret_cast<uint4*>(to + at) = at + 16 <= depth ? __ldg(reinterpret_cast<const uint4*>(row + at)) : last_bytes(row, at, depth);
}

// ---- gradients of few tokens ------------------------------------------------------------------------------------

struct FewGradArgs {
  const void* dout;
  const int8_t* q;                         // w for the input's gradient, x for the weights'
  const float* scale;
  float* part;                             // fp32[splits][tokens][depth]
  void* out;
  int64_t dout_stride, q_stride, out_stride, channels, rows;   // rows: channels of a split
  int tokens, depth, splits;
};

template <class T> __device__ __forceinline__ float as_float(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (__is_same(T, __nv_bfloat16)) return __bfloat162float(v);
  else return __half2float(v);
}

template <class T> __device__ __forceinline__ void put_as(T* p, float v) {
  if constexpr (sizeof(T) == 4) *p = v;
  else if constexpr (__is_same(T, __nv_bfloat16)) *p = __float2bfloat16_rn(v);
  else *p = __float2half_rn(v);
}

// dx of up to TOKENS tokens: a thread holds 8 columns of the weights, a warp 256, a block's eight warps share a split's channels; the
// weights pass once, as they are, a step ahead, and the gradients' few entries times their scales come by way of shared memory.
constexpr int kFewChannels = 32;           // of a step of a block
constexpr int kFewColumns = 256;
// Blocks of an SM: more of them make more parts of dx to join (8 tokens of 85000 x 512: 33 us with 2, 39 with 4), or keep more rows of
// dweight on their way (3 tokens of 67555 x 1078: 77 us with 4, 70 with 8, 63 with 16; 8 tokens of 85000 x 512: 39, 42, 43).
constexpr int64_t kFewBlocks = 2, kFewWeightBlocks = 12;

template <class T, int TOKENS>
__global__ void __launch_bounds__(256) few_input_kernel(const __grid_constant__ FewGradArgs a) {
  pdl_begin();
  constexpr int STEPS = kFewChannels / 8, MINE = (kFewChannels * TOKENS + 255) / 256;
  __shared__ float g[2][kFewChannels][TOKENS];
  __shared__ float joined[8][kFewColumns];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kFewColumns + lane * 8;
  const int64_t first = blockIdx.y * a.rows, last = min(first + a.rows, a.channels);
  float sum[TOKENS][8];
#pragma unroll
  for (int t = 0; t < TOKENS; ++t)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[t][k] = 0.0f;
  uint2 w[STEPS];
  float mine[MINE];
  auto ahead = [&](int64_t n0) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int64_t n = n0 + i * 8 + warp;
      w[i] = make_uint2(0, 0);
      if (n >= last || col >= a.depth) continue;
      const int8_t* p = a.q + n * a.q_stride;
      if (col + 8 <= a.depth) {
        w[i] = __ldg(reinterpret_cast<const uint2*>(p + col));
      } else {
        const uint4 v = last_bytes(p, col, a.depth);
        w[i] = make_uint2(v.x, v.y);
      }
    }
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int at = threadIdx.x + i * 256, t = at / kFewChannels;
      const int64_t n = n0 + at % kFewChannels;
      mine[i] = t < a.tokens && n < last ? as_float<T>(static_cast<const T*>(a.dout)[t * a.dout_stride + n]) * __ldg(a.scale + n) : 0.0f;
    }
  };
  ahead(first);
  int buf = 0;
  for (int64_t n0 = first; n0 < last; n0 += kFewChannels, buf ^= 1) {
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int at = threadIdx.x + i * 256;
      if (at < kFewChannels * TOKENS) g[buf][at % kFewChannels][at / kFewChannels] = mine[i];
    }
    uint2 now[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) now[i] = w[i];
    __syncthreads();                               // (the other half is free: all have left it before they came here)
    if (n0 + kFewChannels < last) ahead(n0 + kFewChannels);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = (float)(int8_t)(now[i].x >> (8 * k));
        v[k + 4] = (float)(int8_t)(now[i].y >> (8 * k));
      }
#pragma unroll
      for (int t = 0; t < TOKENS; ++t) {
        const float f = g[buf][i * 8 + warp][t];
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[t][k] = __fmaf_rn(f, v[k], sum[t][k]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TOKENS; ++t) {
    if (t >= a.tokens) break;
    __syncthreads();
    *reinterpret_cast<float4*>(&joined[warp][lane * 8]) = make_float4(sum[t][0], sum[t][1], sum[t][2], sum[t][3]);
    *reinterpret_cast<float4*>(&joined[warp][lane * 8 + 4]) = make_float4(sum[t][4], sum[t][5], sum[t][6], sum[t][7]);
    __syncthreads();
    const int c = blockIdx.x * kFewColumns + threadIdx.x;
    if (c >= a.depth) continue;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += joined[k][threadIdx.x];
    a.part[((int64_t)blockIdx.y * a.tokens + t) * a.depth + c] = s;
  }
}

// The splits' sums in their order; a warp takes 32 entries of dx, eight warps the splits.
template <class T>
__global__ void __launch_bounds__(256) few_join_kernel(const __grid_constant__ FewGradArgs a) {
  pdl_begin();
  __shared__ float joined[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t all = (int64_t)a.tokens * a.depth, at = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (at < all) {
#pragma unroll 8
    for (int k = warp; k < a.splits; k += 8) s += __ldg(a.part + k * all + at);
  }
  joined[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || at >= all) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += joined[k][lane];
  const int t = (int)(at / a.depth);
  put_as(static_cast<T*>(a.out) + t * a.out_stride + (at - (int64_t)t * a.depth), s);
}

// dweight of up to TOKENS tokens: the call is the weights' way to memory. A thread holds 4 columns of the activations' values and goes
// down its block's channels, whose gradients lie in shared memory; a warp writes 128 entries of a row at a time.
constexpr int kFewRowsAtOnce = 128;

template <class T, int TOKENS, bool VEC>
__global__ void __launch_bounds__(256) few_weight_kernel(const __grid_constant__ FewGradArgs a) {
  pdl_begin();
  __shared__ __align__(16) float g[kFewRowsAtOnce][TOKENS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 128 + (VEC ? lane * 4 : lane), apart = VEC ? 1 : 32;
  float x[TOKENS][4];
#pragma unroll
  for (int t = 0; t < TOKENS; ++t) {
    const float s = t < a.tokens ? __ldg(a.scale + t) : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[t][k] = t < a.tokens && col + k * apart < a.depth ? (float)a.q[t * a.q_stride + col + k * apart] * s : 0.0f;
  }
  const int64_t first = blockIdx.y * a.rows, last = min(first + a.rows, a.channels);
  for (int64_t n0 = first; n0 < last; n0 += kFewRowsAtOnce) {
    __syncthreads();
    for (int i = threadIdx.x; i < kFewRowsAtOnce * TOKENS; i += 256) {
      const int t = i / kFewRowsAtOnce, r = i % kFewRowsAtOnce;
      g[r][t] = t < a.tokens && n0 + r < last ? as_float<T>(static_cast<const T*>(a.dout)[t * a.dout_stride + n0 + r]) : 0.0f;
    }
    __syncthreads();
    const int rows = (int)min((int64_t)kFewRowsAtOnce, last - n0);
#pragma unroll 4
    for (int r = warp; r < rows; r += 8) {
      float v[4];
#pragma unroll
      for (int t = 0; t < TOKENS; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = t == 0 ? g[r][0] * x[0][k] : __fmaf_rn(g[r][t], x[t][k], v[k]);
      float* to = static_cast<float*>(a.out) + (n0 + r) * a.out_stride + col;
      if (VEC && col + 4 <= a.depth) {
        *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (col + k * apart < a.depth) to[k * apart] = v[k];
      }
    }
  }
}

// ---- gradients in parts of bf16 -------------------------------------------------------------------------------

struct OperandArgs {
  const void* dout;
  __nv_bfloat16* a;                        // its planes, or null: its rows are read as they are
  const int8_t* q;
  const float* scale;
  __nv_bfloat16* b;
  int64_t dout_stride, a_stride, tokens, channels, q_stride, b_stride, along;
  int depth, a_blocks;                     // blocks of the grid that make the planes
};

// 8 entries of x as a sum of PLANES bf16 numbers each, exact (8 bits of the significand in each): the first holds what is no number.
template <class T, int PLANES>
__device__ __forceinline__ void planes(const OperandArgs& a, int64_t block, int64_t blocks) {
  const int64_t per = (a.channels + 7) / 8;
  for (int64_t i = block * blockDim.x + threadIdx.x; i < a.tokens * per; i += blocks * blockDim.x) {
    const int64_t row = i / per, at = (i - row * per) * 8;
    const T* p = static_cast<const T*>(a.dout) + row * a.dout_stride + at;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = at + k < a.channels ? as_float<T>(p[k]) : 0.0f;
#pragma unroll
    for (int plane = 0; plane < PLANES; ++plane) {
      __nv_bfloat16 e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t bits = __float_as_uint(v[k]);
        if ((bits & 0x7f800000u) == 0x7f800000u) {             // infinite: only here; NaN stays one
          e[k] = __float2bfloat16_rn(v[k]);
          v[k] = 0.0f;
        } else {
          const float high = __uint_as_float(bits & 0xffff0000u);
          e[k] = __float2bfloat16_rn(high);
          v[k] -= high;
        }
      }
      *reinterpret_cast<uint4*>(a.a + ((int64_t)plane * a.tokens + row) * a.a_stride + at) = *reinterpret_cast<const uint4*>(e);
    }
  }
}

// What a gradient's tiles read, in one launch: the planes of dout, and the values of the rows in 8 bits.
template <class T, int PLANES>
__global__ void __launch_bounds__(256) operands_kernel(const __grid_constant__ OperandArgs a) {
  pdl_begin();
  if ((int)blockIdx.x < a.a_blocks) {
    planes<T, PLANES>(a, blockIdx.x, a.a_blocks);
    return;
  }
  const int64_t per = (a.depth + 15) / 16, blocks = gridDim.x - a.a_blocks;
  for (int64_t i = (int64_t)(blockIdx.x - a.a_blocks) * blockDim.x + threadIdx.x; i < a.along * per; i += blocks * blockDim.x) {
    const int64_t row = i / per;
    const int at = (int)(i - row * per) * 16;
    const float s = __ldg(a.scale + row);
    const int8_t* p = a.q + row * a.q_stride;
    const uint4 raw = at + 16 <= a.depth ? __ldg(reinterpret_cast<const uint4*>(p + at)) : last_bytes(p, at, a.depth);
    const int8_t* b = reinterpret_cast<const int8_t*>(&raw);
    __nv_bfloat16 v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __float2bfloat16_rn((float)b[k] * s);
    uint4* to = reinterpret_cast<uint4*>(a.b + row * a.b_stride + at);
    to[0] = reinterpret_cast<const uint4*>(v)[0];
    if (at + 8 < a.b_stride) to[1] = reinterpret_cast<const uint4*>(v)[1];
  }
}

// ---- host ----------------------------------------------------------------------------------------------------------

bool known(int32_t t) { return t == GSPARSE_F32 || t == GSPARSE_BF16 || t == GSPARSE_F16; }
size_t size_of(int32_t t) { return t == GSPARSE_F32 ? 4 : 2; }
bool at_multiple(const void* p, size_t of) { return (reinterpret_cast<uintptr_t>(p) % of) == 0; }

int sizes(int64_t tokens, int64_t channels, int64_t depth) {
  if (tokens < 0 || channels < 1 || depth < 1) return GSPARSE_ERR_INVALID_ARG;
  if (tokens > GSPARSE_MAX_ROWS || channels > GSPARSE_MAX_ROWS || depth > GSPARSE_MAX_DEPTH) return GSPARSE_ERR_UNSUPPORTED;
  return GSPARSE_OK;
}

bool rows8(const int8_t* q, int64_t stride, const float* scale, int64_t depth) {
  return q && scale && aligned16(q) && stride % 16 == 0 && stride >= depth && at_multiple(scale, 4);
}

bool matrix(const void* p, int64_t stride, int32_t dtype, int64_t rows, int64_t cols, bool write) {
  return known(dtype) && p && at_multiple(p, size_of(dtype)) && stride >= (write && rows > 1 ? cols : 0);
}

bool space(const void* workspace, size_t have, size_t need) { return workspace && at_multiple(workspace, 256) && have >= need; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess) {
      cudaGetLastError();
      return (EncodeTiled) nullptr;
    }
    return r == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(p) : nullptr;
  }();
  return f;
}

// Rows of 8-, 16- or 32-bit entries, `stride` entries apart, in `planes` matrices one after another; boxes of 128 bytes by `high` rows.
bool map_of(CUtensorMap* m, CUtensorMapDataType type, int bytes, const void* p, int64_t cols, int64_t rows, int64_t stride, int high,
            int planes = 0) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const int64_t step = (rows > 1 ? stride : round_up(cols, 16 / bytes)) * bytes;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(planes ? planes : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)step, (cuuint64_t)(step * rows)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / bytes), (cuuint32_t)high, 1}, one[3] = {1, 1, 1};
  return encode(m, type, planes ? 3 : 2, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

CUtensorMapDataType map_type(int32_t dtype) {
  return dtype == GSPARSE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : dtype == GSPARSE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// How the tiles of D are shared out: whole tiles in waves over the pairs of SMs; what is left over is split along s.
// Tiles side by side: 16 of the product (8192 x 32003 x 4096: 754 us, 8: 775), 8 of the gradients (4000 x 85000 x 512: 313, 16: 318).
constexpr int kProductBand = 16, kGradBand = 8;
// Bytes of an operand that the second-level cache may be asked to keep (of 126 MB), while the other passes once: gradient by the weights
// of 85000 x 512 over 4000 tokens 313 us, without either hint 361 (long runs).
constexpr int64_t kKeep = 96 << 20;

int64_t part_entries(const Plan& p) { return p.piece ? 2 * (int64_t)p.pairs * kTile * kTile : 0; }

constexpr int64_t kFewTokens = 4;          // (8 tokens against 85000 x 512: 34 us there, 4: 16; the tiles take 17)

template <int TOKENS, int ROWS>
void few_of(const FewArgs& a, cudaStream_t st) {
  // Channels for fewer than 32 warps on each SM, and a depth that leaves every warp of a block something: split (a token of
  // 1000 x 2048: 2.5 us, 3.1 without; of 85000 x 512, which is not: 10).
  const bool split = a.channels < (int64_t)ROWS * 32 * sm_count() && a.depth >= 1024;
  const dim3 grid((unsigned)cdiv(a.channels, split ? ROWS : 8 * ROWS));
  if (split) launch(few_kernel<TOKENS, ROWS, true>, grid, dim3(256), 0, st, a);
  else launch(few_kernel<TOKENS, ROWS, false>, grid, dim3(256), 0, st, a);
}

int few(const FewArgs& a, cudaStream_t st) {
  if (a.tokens == 1) few_of<1, 4>(a, st);
  else if (a.tokens == 2) few_of<2, 4>(a, st);
  else few_of<4, 4>(a, st);
  return launch_status();
}

bool fits(int64_t rows, int64_t cols) { return cdiv(rows, kTile) * cdiv(cols, kTile) < (1ll << 30); }

template <bool INT, int WARPS>
void join_of(const JoinArgs& j, int tiles, int32_t dtype, cudaStream_t st) {
  const dim3 grid((unsigned)(32 * WARPS * tiles));
  if (dtype == GSPARSE_F32) launch(join_kernel<INT, float, WARPS>, grid, dim3(256), 0, st, j);
  else if (dtype == GSPARSE_BF16) launch(join_kernel<INT, __nv_bfloat16, WARPS>, grid, dim3(256), 0, st, j);
  else launch(join_kernel<INT, __half, WARPS>, grid, dim3(256), 0, st, j);
}

template <bool INT, bool A_ACROSS>
int tiles(TileArgs& a, const Plan& p, float* part, void* out, int64_t out_stride, cudaStream_t st) {
  a.order = p.order;
  a.blocks = p.blocks;
  a.pairs = p.pairs;
  a.waves = p.waves;
  a.piece = p.piece;
  a.group = p.group;
  a.span = p.span;
  using L = Layout<INT>;
  const int32_t dtype = a.out_dtype;
  const int bytes = (int)size_of(dtype);
  const bool as_tiles = aligned16(out) && (a.rows == 1 || (out_stride * bytes) % 16 == 0);
  a.result = out;
  a.result_stride = out_stride;
  a.as_tiles = as_tiles ? a.cols / (16 / bytes) * (16 / bytes) : 0;
  if (a.as_tiles && !map_of(&a.out, map_type(dtype), bytes, out, a.as_tiles, a.rows, out_stride, 32)) return GSPARSE_ERR_CUDA;
  if (p.piece && !map_of(&a.part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, part, kTile, 2 * (int64_t)p.pairs * kTile, kTile, 32)) return GSPARSE_ERR_CUDA;
  auto* kernel = tile_kernel<INT, A_ACROSS>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::shared) != cudaSuccess) {
    cudaGetLastError();
    return GSPARSE_ERR_CUDA;
  }
  const int used = p.piece || p.waves ? p.pairs : p.tiles;
  launch(kernel, dim3((unsigned)(2 * used)), dim3(L::threads), L::shared, st, (const TileArgs&)a);
  if (p.piece) {
    JoinArgs j{part, a.row_scale, a.col_scale, out, out_stride, a.rows, a.cols, p.order, p.waves * p.pairs, p.blocks, p.piece, p.group, p.span, 1, 0};
    if (a.stacked) {
      j.planes = a.stacked;
      j.rows = a.rows / a.stacked;
      j.plane_rows = (int)j.rows;
    }
    const int parts = (int)cdiv(p.blocks, p.piece) * j.planes;
    // (5 parts a row, 184 x 1373 x 3872 fp32: 29 us with a warp a row, 33 with eight; 33 parts, 88 x 8383 x 103: 28 and 14)
    if (parts > 8) join_of<INT, 8>(j, p.tiles - p.waves * p.pairs, dtype, st);
    else join_of<INT, 1>(j, p.tiles - p.waves * p.pairs, dtype, st);
  }
  return launch_status();
}

// What the product keeps in the workspace.
struct Product {
  Plan plan;
  int copies;
  int8_t* copy;
  float* part;
  size_t bytes;
};

Product product_of(void* workspace, int64_t tokens, int64_t channels, int64_t depth) {
  Product p{};
  if (tokens <= kFewTokens) return p;
  p.plan = plan_of(tokens, channels, cdiv(depth, 128), kProductBand, sm_count() / 2);
  const int64_t x = tokens * round_up(depth, 16);
  Carver c(workspace);
  p.copies = x <= kCopyBytes ? (int)min(cdiv(kCopiesBytes, x), (int64_t)p.plan.pairs) : 1;
  if (p.copies > 1) p.copy = c.take<int8_t>(p.copies * x);
  if (part_entries(p.plan)) p.part = c.take<float>(part_entries(p.plan));
  p.bytes = c.off;
  return p;
}

// Gradients of few tokens: a block takes some columns and a split of the channels.
FewGradArgs few_grad(const void* dout, int64_t dout_stride, const int8_t* q, int64_t q_stride, const float* scale, int64_t tokens, int64_t channels,
                     int64_t depth, bool weight) {
  FewGradArgs a{dout, q, scale, nullptr, nullptr, dout_stride, q_stride, 0, channels, 0, (int)tokens, (int)depth, 0};
  const int64_t across = cdiv(depth, weight ? 128 : kFewColumns), want = cdiv((weight ? kFewWeightBlocks : kFewBlocks) * sm_count(), across);
  a.rows = round_up(cdiv(channels, want), kFewChannels);
  a.splits = (int)cdiv(channels, a.rows);
  return a;
}

template <class T>
void few_input_of(const FewGradArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)cdiv(a.depth, kFewColumns), (unsigned)a.splits);
  if (a.tokens <= 1) launch(few_input_kernel<T, 1>, grid, dim3(256), 0, st, a);
  else if (a.tokens <= 2) launch(few_input_kernel<T, 2>, grid, dim3(256), 0, st, a);
  else if (a.tokens <= 4) launch(few_input_kernel<T, 4>, grid, dim3(256), 0, st, a);
  else launch(few_input_kernel<T, 8>, grid, dim3(256), 0, st, a);
}

template <class T, bool VEC>
void few_weight_of(const FewGradArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)cdiv(a.depth, 128), (unsigned)a.splits);
  if (a.tokens <= 1) launch(few_weight_kernel<T, 1, VEC>, grid, dim3(256), 0, st, a);
  else if (a.tokens <= 2) launch(few_weight_kernel<T, 2, VEC>, grid, dim3(256), 0, st, a);
  else if (a.tokens <= 4) launch(few_weight_kernel<T, 4, VEC>, grid, dim3(256), 0, st, a);
  else launch(few_weight_kernel<T, 8, VEC>, grid, dim3(256), 0, st, a);
}

// (8 tokens of 85000 x 512 bf16: dx 33 us and 64 in the tiles, dweight 42 and 38; of 1000 x 2048: 6 and 27, 8 and 12)
constexpr int64_t kFewGradTokens = 8;

int few_gradient(bool weight, FewGradArgs a, int32_t dtype, void* out, int32_t out_dtype, int64_t out_stride, float* part, cudaStream_t st) {
  a.out = out;
  a.out_stride = out_stride;
  a.part = part;
  if (weight) {
    const bool vec = aligned16(out) && (a.channels == 1 || out_stride % 4 == 0);
    if (dtype == GSPARSE_F32) vec ? few_weight_of<float, true>(a, st) : few_weight_of<float, false>(a, st);
    else if (dtype == GSPARSE_BF16) vec ? few_weight_of<__nv_bfloat16, true>(a, st) : few_weight_of<__nv_bfloat16, false>(a, st);
    else vec ? few_weight_of<__half, true>(a, st) : few_weight_of<__half, false>(a, st);
    return launch_status();
  }
  if (dtype == GSPARSE_F32) few_input_of<float>(a, st);
  else if (dtype == GSPARSE_BF16) few_input_of<__nv_bfloat16>(a, st);
  else few_input_of<__half>(a, st);
  const dim3 grid((unsigned)cdiv((int64_t)a.tokens * a.depth, 32));
  if (out_dtype == GSPARSE_F32) launch(few_join_kernel<float>, grid, dim3(256), 0, st, (const FewGradArgs&)a);
  else if (out_dtype == GSPARSE_BF16) launch(few_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, (const FewGradArgs&)a);
  else launch(few_join_kernel<__half>, grid, dim3(256), 0, st, (const FewGradArgs&)a);
  return launch_status();
}

// A gradient's operands in the workspace: dout in planes of bf16 where it is not bf16 rows at 16-byte boundaries already, and the
// values of the rows in 8 bits.
struct Grad {
  Plan plan;
  bool stacked;
  int planes;
  bool copied;
  int64_t stride_a, stride_b;
  __nv_bfloat16* a;
  __nv_bfloat16* b;
  float* part;
  size_t bytes;
};

Grad grad_of(void* workspace, const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens, int64_t channels, int64_t depth, bool weight) {
  Grad g{};
  g.planes = dtype == GSPARSE_F32 ? 3 : dtype == GSPARSE_F16 ? 2 : 1;
  g.copied = dtype != GSPARSE_BF16 || !aligned16(dout) || (tokens > 1 && (dout_stride % 8 || dout_stride < channels));
  g.stride_a = round_up(channels, 8);
  g.stride_b = round_up(depth, 8);
  Carver c(workspace);
  if (tokens <= kFewGradTokens) {
    if (!weight) g.part = c.take<float>(few_grad(dout, 0, nullptr, 0, nullptr, tokens, channels, depth, false).splits * tokens * depth);
    g.bytes = c.off;
    return g;
  }
  g.a = c.take<__nv_bfloat16>(g.copied ? g.planes * tokens * g.stride_a : 0);
  const int64_t along = weight ? tokens : channels;
  g.b = c.take<__nv_bfloat16>(along * g.stride_b);
  // The planes of few tokens as rows of one tile: the weights are read once, not once a plane.
  g.stacked = !weight && g.planes > 1 && g.planes * tokens <= kTile && cdiv(depth, kTile) <= sm_count() / 2;
  const int pairs = sm_count() / 2;
  const Plan& p = g.plan = g.stacked ? plan_of(g.planes * tokens, depth, cdiv(along, 64), kGradBand, pairs, true)
                                     : plan_of(weight ? channels : tokens, depth, g.planes * cdiv(along, 64), kGradBand, pairs);
  g.part = c.take<float>(part_entries(p));
  g.bytes = c.off + 256;
  return g;
}

size_t grad_bytes(const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens, int64_t channels, int64_t depth, bool weight) {
  if (!known(dtype) || sizes(tokens, channels, depth) != GSPARSE_OK || !fits(weight ? channels : tokens, depth)) return 0;
  return grad_of(nullptr, dout, dtype, dout_stride, tokens, channels, depth, weight).bytes;
}

bool grad_space(const void* workspace, size_t have, const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens, int64_t channels,
                int64_t depth, bool weight) {
  const size_t need = grad_bytes(dout, dtype, dout_stride, tokens, channels, depth, weight);
  return !need || space(workspace, have, need);
}

// Blocks of 64 products that the matrix unit adds before they are rounded to the nearest: it cuts off, so that C products in a row are
// off by about C 1.3e-9 of the sum, in one direction. A plain fp32 product's error grows with the root of the sum's length S (S = 256:
// 2.1e-7, 1000: 5.2e-7, 4000: 1.06e-6, 2-norms against 64 bits); C keeps to it: 128 (1.8e-7) for up to 7 blocks, 256 (3.4e-7) for up
// to 31 and for gradients in fp32, 512 (6.4e-7) for the others. Results of 16 bits take 512 from 8 blocks on (4000 x 85000 x 512 bf16 by the
// input 297 us, 291 with 2048, and 4000 x 1900 x 4096 55 us, 60 with 256; by the weights 1000 x 8192 x 4096 68 us with 256, 65 with 512; 500
// tokens 53 with 128, 43 with 256; 2000 x 400 x 2048 by the input 12.4 with 128 as with 512).
int chunk_of(int32_t dtype, int32_t out_dtype, int blocks) {
  const int chunk = blocks < 8 ? 2 : blocks < 32 && out_dtype == GSPARSE_F32 ? 4 : 8;
  return dtype == GSPARSE_F32 && chunk > 4 ? 4 : chunk;
}

template <bool WEIGHT>
int gradient(const void* dout, int32_t dtype, int64_t dout_stride, const int8_t* q, int64_t q_stride, const float* scale, int64_t tokens,
             int64_t channels, int64_t depth, void* out, int32_t out_dtype, int64_t out_stride, void* workspace, int32_t* d_status,
             cudaStream_t st) {
  const Grad g = grad_of(workspace, dout, dtype, dout_stride, tokens, channels, depth, WEIGHT);
  const int64_t along = WEIGHT ? tokens : channels;
  if (tokens <= kFewGradTokens)
    return few_gradient(WEIGHT, few_grad(dout, dout_stride, q, q_stride, scale, tokens, channels, depth, WEIGHT), dtype, out, out_dtype, out_stride, g.part,
                        st);
  OperandArgs o{dout, g.a, q, scale, g.b, dout_stride, g.stride_a, tokens, channels, q_stride, g.stride_b, along, (int)depth, 0};
  auto blocks_of = [](int64_t vectors) {
    const int64_t need = cdiv(vectors, 256), most = (int64_t)sm_count() * 16;
    return (int)(need < most ? need : most);
  };
  if (g.copied) o.a_blocks = blocks_of(tokens * cdiv(channels, 8));
  const dim3 grid((unsigned)(o.a_blocks + blocks_of(along * cdiv(depth, 16))));
  if (dtype == GSPARSE_F32) launch(operands_kernel<float, 3>, grid, dim3(256), 0, st, (const OperandArgs&)o);
  else if (dtype == GSPARSE_F16) launch(operands_kernel<__half, 2>, grid, dim3(256), 0, st, (const OperandArgs&)o);
  else launch(operands_kernel<__nv_bfloat16, 1>, grid, dim3(256), 0, st, (const OperandArgs&)o);
  TileArgs a{};
  if (!map_of(&a.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.copied ? g.a : dout, channels, g.stacked ? g.planes * tokens : tokens,
              g.copied ? g.stride_a : dout_stride, WEIGHT ? 64 : 128, g.stacked ? 1 : g.planes) ||
      !map_of(&a.b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.b, depth, along, g.stride_b, 64))
    return GSPARSE_ERR_CUDA;
  a.d_status = d_status;
  a.stacked = g.stacked ? g.planes : 0;
  a.rows = WEIGHT ? channels : g.stacked ? g.planes * tokens : tokens;
  a.cols = depth;
  a.plane_blocks = (int)cdiv(along, 64);
  a.out_dtype = out_dtype;
  a.chunk = chunk_of(dtype, out_dtype, a.plane_blocks);
  const Plan& p = g.plan;
  a.keep_a = p.order.bands == 1 && !p.order.wide ? -1 : 0;    // the tiles of a row of them are under way together
  a.keep_b = along * g.stride_b * 2 <= kKeep ? 1 : 0;
  return tiles<false, WEIGHT>(a, p, g.part, out, out_stride, st);
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" {

size_t gsparse_linear_q8_workspace_size(int64_t tokens, int64_t channels, int64_t depth) {
  if (sizes(tokens, channels, depth) != GSPARSE_OK || !fits(tokens, channels)) return 0;
  return product_of(nullptr, tokens, channels, depth).bytes;
}

int gsparse_linear_q8(const int8_t* x, int64_t x_stride, const float* x_scale, const int8_t* w, int64_t w_stride, const float* w_scale,
                      int64_t tokens, int64_t channels, int64_t depth, void* out, int32_t dtype, int64_t out_stride, void* workspace,
                      size_t workspace_bytes, int32_t* d_status, gsparse_stream stream) {
  const int st = sizes(tokens, channels, depth);
  if (st != GSPARSE_OK) return st;
  if (!fits(tokens, channels)) return GSPARSE_ERR_UNSUPPORTED;
  if (!known(dtype)) return GSPARSE_ERR_INVALID_ARG;
  if (tokens == 0) return GSPARSE_OK;
  if (!rows8(x, x_stride, x_scale, depth) || !rows8(w, w_stride, w_scale, depth) || !matrix(out, out_stride, dtype, tokens, channels, true))
    return GSPARSE_ERR_INVALID_ARG;
  const Product p = product_of(workspace, tokens, channels, depth);
  if (p.bytes && !space(workspace, workspace_bytes, p.bytes)) return GSPARSE_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if (tokens <= kFewTokens)
    return few({x, w, x_scale, w_scale, out, x_stride, w_stride, out_stride, channels, (int)tokens, (int)depth, dtype}, s);
  const int64_t copy_stride = round_up(depth, 16);
  if (p.copy)
    launch(copies_kernel, dim3((unsigned)(p.copies * tokens)), dim3(128), 0, s, x, x_stride, (int)tokens, (int)depth, p.copy, copy_stride);
  TileArgs a{};
  if (!map_of(&a.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.copy ? p.copy : x, depth, tokens, p.copy ? copy_stride : x_stride, 128, p.copies) ||
      !map_of(&a.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, depth, channels, w_stride, 128))
    return GSPARSE_ERR_CUDA;
  a.copies = p.copies;
  a.row_scale = x_scale;
  a.col_scale = w_scale;
  a.d_status = d_status;
  a.rows = tokens;
  a.cols = channels;
  a.plane_blocks = (int)cdiv(depth, 128);
  a.out_dtype = dtype;
  return tiles<true, false>(a, p.plan, p.part, out, out_stride, s);
}

size_t gsparse_linear_q8_grad_input_workspace_size(const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens,
                                                   int64_t channels, int64_t depth) {
  return grad_bytes(dout, dtype, dout_stride, tokens, channels, depth, false);
}

int gsparse_linear_q8_grad_input(const void* dout, int32_t dtype, int64_t dout_stride, const int8_t* w, int64_t w_stride,
                                 const float* w_scale, int64_t tokens, int64_t channels, int64_t depth, void* dx, int32_t dx_dtype,
                                 int64_t dx_stride, void* workspace, size_t workspace_bytes, int32_t* d_status, gsparse_stream stream) {
  const int st = sizes(tokens, channels, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(dtype) || !known(dx_dtype)) return GSPARSE_ERR_INVALID_ARG;
  if (tokens == 0) return GSPARSE_OK;
  if (!matrix(dout, dout_stride, dtype, tokens, channels, false) || !rows8(w, w_stride, w_scale, depth) ||
      !matrix(dx, dx_stride, dx_dtype, tokens, depth, true))
    return GSPARSE_ERR_INVALID_ARG;
  if (!grad_space(workspace, workspace_bytes, dout, dtype, dout_stride, tokens, channels, depth, false)) return GSPARSE_ERR_WORKSPACE;
  return gradient<false>(dout, dtype, dout_stride, w, w_stride, w_scale, tokens, channels, depth, dx, dx_dtype, dx_stride, workspace, d_status,
                         (cudaStream_t)stream);
}

size_t gsparse_linear_q8_grad_weight_workspace_size(const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens,
                                                    int64_t channels, int64_t depth) {
  return grad_bytes(dout, dtype, dout_stride, tokens, channels, depth, true);
}

int gsparse_linear_q8_grad_weight(const void* dout, int32_t dtype, int64_t dout_stride, const int8_t* x, int64_t x_stride,
                                  const float* x_scale, int64_t tokens, int64_t channels, int64_t depth, float* dweight,
                                  int64_t dweight_stride, void* workspace, size_t workspace_bytes, int32_t* d_status,
                                  gsparse_stream stream) {
  const int st = sizes(tokens, channels, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(dtype) || !matrix(dweight, dweight_stride, GSPARSE_F32, channels, depth, true)) return GSPARSE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (tokens == 0) {
    if (cudaMemset2DAsync(dweight, (size_t)(channels > 1 ? dweight_stride : depth) * 4, 0, (size_t)depth * 4, (size_t)channels, s) != cudaSuccess) {
      cudaGetLastError();
      return GSPARSE_ERR_CUDA;
    }
    return GSPARSE_OK;
  }
  if (!matrix(dout, dout_stride, dtype, tokens, channels, false) || !rows8(x, x_stride, x_scale, depth)) return GSPARSE_ERR_INVALID_ARG;
  if (!grad_space(workspace, workspace_bytes, dout, dtype, dout_stride, tokens, channels, depth, true)) return GSPARSE_ERR_WORKSPACE;
  return gradient<true>(dout, dtype, dout_stride, x, x_stride, x_scale, tokens, channels, depth, dweight, GSPARSE_F32, dweight_stride, workspace,
                        d_status, s);
}

}  // extern "C"

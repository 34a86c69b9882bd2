// What the two kernels of grouped MX products share: the groups' tiles, the
// scales' layout for the tensor cores, issue by one lane of a converged warp.
#pragma once

#include <mutex>

#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "mx_format.cuh"

namespace rmoe {

constexpr int MX_SF_BYTES = 512;    // scale words of 128 operand rows, one K step's word
constexpr int MX_MAX_GROUPS = 128;
constexpr unsigned FULL = 0xffffffffu;

// Wait for a phase without regard to the abort flag, bounded by timeout_ns.
__device__ __forceinline__ void mbar_wait_drain(uint64_t* bar, uint32_t parity,
                                                uint64_t timeout_ns) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (globaltimer_ns() - t0 > timeout_ns) return;
  }
}

// A value that is the same in all lanes, told to the compiler, which then keeps
// it (and branches on it) in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(FULL, v, 0); }

struct Tile {
  int g, row0, rows, nt;
};

// The tiles (of TILE rows) of one CTA or cluster in order: every n-th, columns
// fastest.  The warp finds the next one's group together (32 groups a look).
template <int TILE>
struct TileWalk {
  int g, mt, nt;

  __device__ __forceinline__ void start(int tile, int n_tiles, int groups, const int* mts) {
    mt = tile / n_tiles;
    nt = tile - mt * n_tiles;
    g = 0;
    seek(groups, mts);
  }
  __device__ __forceinline__ void next(int dm, int dn, int n_tiles, int groups, const int* mts) {
    mt += dm;
    nt += dn;
    if (nt >= n_tiles) {
      nt -= n_tiles;
      ++mt;
    }
    seek(groups, mts);
  }
  // largest g with mts[g] <= mt (skips empty groups); g is never past it
  __device__ __forceinline__ void seek(int groups, const int* mts) {
    unsigned b;
    do {
      const int i = min(g + (int)(threadIdx.x & 31), groups);
      b = __ballot_sync(FULL, mts[i] <= mt && i < groups);
      g += __popc(b) - 1;
    } while (b == FULL);
  }
  __device__ __forceinline__ Tile tile(const int* mts, const int* rs) const {
    Tile t;
    t.g = g;
    t.nt = nt;
    t.row0 = uniform(rs[g] + (mt - mts[g]) * TILE);
    t.rows = min(TILE, uniform(rs[g + 1]) - t.row0);
    return t;
  }
};

// The same expression as in the bf16 kernels.
__device__ __forceinline__ float silu_f(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

// Rows of groups and the prefix of their tiles, from the caller's offsets.
// Offsets outside the rows are cut to them and ones that run backwards raised to
// the largest before them, so that no access leaves the operands; both are
// reported.
struct MxGroups {
  int mt_start[MX_MAX_GROUPS + 1];
  int row_start[MX_MAX_GROUPS + 1];
};

// All threads of the block; returns the number of row tiles.
template <int TILE>
__device__ __forceinline__ int mx_group_table(const MxGemmArgs& a, MxGroups& t) {
  if (threadIdx.x < 32) {  // 5 offsets per lane
    constexpr int PER = MX_MAX_GROUPS / 32 + 1;
    const int lane = threadIdx.x;
    if (lane == 0 && blockIdx.x == 0 && a.clear_status) {
      a.status[0] = 0;
      a.status[1] = 0;
    }
    int at[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int g = lane * PER + q;
      at[q] = a.offsets[min(g, a.groups)];
    }
    int prev = __shfl_up_sync(FULL, at[PER - 1], 1);  // the offset before this lane's
    if (lane == 0) prev = 0;
    bool bad = false;
    int low = prev;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      bad |= at[q] < low || at[q] > a.rows;
      low = at[q];
    }
    if (__any_sync(FULL, bad)) {
      if (lane == 0 && blockIdx.x == 0) report_error(a.status, MOE_ERR_DEVICE_INDEX, 60);
      int top = 0;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        top = max(top, min(at[q], a.rows));
        at[q] = top;
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(FULL, top, off);
        if (lane >= off) top = max(top, u);
      }
      prev = __shfl_up_sync(FULL, top, 1);
      if (lane == 0) prev = 0;
#pragma unroll
      for (int q = 0; q < PER; ++q) at[q] = max(at[q], prev);
    }
    int loc[PER], sum = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {  // loc: tiles of group g - 1
      const int g = lane * PER + q;
      if (g <= a.groups) t.row_start[g] = at[q];
      loc[q] = g > 0 && g <= a.groups ? (at[q] - prev + TILE - 1) / TILE : 0;
      sum += loc[q];
      prev = at[q];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(FULL, incl, off);
      if (lane >= off) incl += u;
    }
    int run = incl - sum;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int g = lane * PER + q;
      run += loc[q];
      if (g <= a.groups) t.mt_start[g] = run;
    }
  }
  __syncthreads();
  return t.mt_start[a.groups];
}

// Instruction descriptor without the scale ids: UE8M0 scales.
template <int FMT>
__device__ __forceinline__ constexpr uint32_t idesc_mx(int M, int N) {
  return (FMT == MOE_MXFP4 ? (1u << 7) | (1u << 10) : 0u)  // E2M1 (0: E4M3)
         | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// MMA kk of a K step uses scale byte kk (MXFP8) or bytes 2*(kk%2).. (MXFP4).
__device__ __forceinline__ uint32_t idesc_sf(uint32_t idesc, uint32_t id) {
  return idesc | (id << 4) | (id << 29);
}

// Unswizzled rows of 16 bytes: 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_rows16(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Named barrier of N warps that work together (id 1..15).
template <int N>
__device__ __forceinline__ void warps_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(32 * N) : "memory");
}

// The same, and whether ok holds in all of them.
template <int N>
__device__ __forceinline__ bool warps_agree(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, r;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "bar.red.and.pred r, %1, %3, p;\n\tselp.u32 %0, 1, 0, r;\n\t}\n"
      : "=r"(all)
      : "r"(id), "r"(static_cast<uint32_t>(ok)), "n"(32 * N)
      : "memory");
  return all != 0;
}

// Shared memory to global memory (16-byte aligned, whole 16 bytes), part of this
// thread's open group of copies.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}

// ---------------------------------------------------------------- host
inline PFN_cuTensorMapEncodeTiled_v12000 mx_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

inline cudaError_t encode_tmap(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                   CUtensorMapSwizzle swizzle) {
  auto fn = mx_encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_in_context([&] {
    return fn(map, type, rank, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

}  // namespace rmoe

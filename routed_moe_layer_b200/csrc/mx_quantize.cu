// Quantisation to the MX formats and back, and the RMSNorm whose output is
// quantised (formats and rounding: mx_format.cuh).
//
// All three move each value once and compute a handful of operations on it, so
// HBM bounds them: 2 B read + 1.03 B (MXFP8) or 0.53 B (MXFP4) written a value
// for the quantisation, the reverse for its inverse, and 4 B read + 4 B + 1.03 B
// written for the norm with a residual.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mx_format.cuh"

namespace rmoe {

namespace {

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t pair) {
  return __vmaxu2(m, pair & 0x7fff7fffu);
}

// Largest |v| of a pair of bf16 magnitudes, as fp32 bits.
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) { return max(m & 0xffffu, m >> 16) << 16; }

// 32 bytes (16 bf16) as one load / store; the address must be 32-byte aligned.
__device__ __forceinline__ void load_v8(const void* src, uint32_t (&v)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                 "=r"(v[6]), "=r"(v[7])
               : "l"(src));
}

// Quantisation and its inverse share their layout: eight lanes hold 128
// consecutive elements of a row (a word of scales), 16 each, two lanes to a
// block; a warp covers four rows, whose words are 16 consecutive bytes, and
// U words of each, all loaded before the first is used.  blockIdx.y counts
// groups of U words.  K past the row's end counts as nothing: no
// load, no codes, a zero scale byte.
//
// 24,576 x 2048 to MXFP8: 25.1 us (6.1 TB/s, 0.94 of the measured copy); one word
// a lane 26.0.  240 x 1024 to MXFP4 and back: one word a lane 2.9 us, four 4.1
// (too few warps to hide the memory's latency), so calls that would not put 8
// blocks on every SM take one.

struct MxPlace {
  long long row;        // row of all matrices
  long long word0;      // index of word 0 of the row
  int k0;               // this lane's first element of the first word
  int sub;              // lane of the eight
  bool live;
};

template <int U>
__device__ __forceinline__ MxPlace mx_place(long long total_rows, int rows, int words) {
  MxPlace p;
  const int lane = threadIdx.x & 31;
  p.sub = lane & 7;
  p.row = ((long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  p.live = p.row < total_rows;
  const long long g = total_rows > rows ? p.row / rows : 0;
  p.word0 = g * words * rows + (p.row - g * rows);
  p.k0 = (int)blockIdx.y * U * 128 + p.sub * 16;
  return p;
}

template <int FMT, int U>
__global__ void __launch_bounds__(256)
    mx_quantize_kernel(const __nv_bfloat16* __restrict__ x, long long total_rows, int rows, int K,
                       int words, uint8_t* __restrict__ codes, uint32_t* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  const MxPlace p = mx_place<U>(total_rows, rows, words);
  uint32_t v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (p.live && p.k0 + 128 * u < K)
      load_v8(x + p.row * K + p.k0 + 128 * u, v[u]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = p.k0 + 128 * u;
    const bool live = p.live && k < K;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = abs_max2(m, v[u][i]);
    m = abs_max2(m, __shfl_xor_sync(FULL, m, 1));
    const uint32_t byte = mx_scale_byte<FMT>(amax_bits(m));
    uint32_t word = live ? byte << (8 * (p.sub >> 1)) : 0;
    word |= __shfl_xor_sync(FULL, word, 2);
    word |= __shfl_xor_sync(FULL, word, 4);
    if (live) {
      float f[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[2 * i] = bf16_lo(v[u][i]);
        f[2 * i + 1] = bf16_hi(v[u][i]);
      }
      uint32_t o[4];
      mx_encode<FMT>(f, byte, o);
      if constexpr (FMT == MOE_MXFP8)
        *reinterpret_cast<uint4*>(codes + p.row * K + k) = make_uint4(o[0], o[1], o[2], o[3]);
      else
        *reinterpret_cast<uint2*>(codes + (p.row * K + k) / 2) = make_uint2(o[0], o[1]);
      if (p.sub == 0) scales[p.word0 + (long long)(k >> 7) * rows] = word;
    }
  }
}

template <int FMT, int U>
__global__ void __launch_bounds__(256)
    mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint32_t* __restrict__ scales,
                         long long total_rows, int rows, int K, int words,
                         __nv_bfloat16* __restrict__ x) {
  pdl_launch_dependents();
  pdl_wait();
  const MxPlace p = mx_place<U>(total_rows, rows, words);
  if (!p.live) return;
  constexpr int CW = FMT == MOE_MXFP8 ? 4 : 2;  // words of 16 codes
  uint32_t c[U][4], sw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = p.k0 + 128 * u;
    if (k < K) {
      if constexpr (FMT == MOE_MXFP8)
        *reinterpret_cast<uint4*>(c[u]) = *reinterpret_cast<const uint4*>(codes + p.row * K + k);
      else
        *reinterpret_cast<uint2*>(c[u]) =
            *reinterpret_cast<const uint2*>(codes + (p.row * K + k) / 2);
      sw[u] = scales[p.word0 + (long long)(k >> 7) * rows];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = p.k0 + 128 * u;
    if (k < K) {
      const float s = mx_scale_value((sw[u] >> (8 * (p.sub >> 1))) & 0xffu);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f;
        if constexpr (FMT == MOE_MXFP8)
          f = mx_unpack_e4m3((c[u][i * CW / 8] >> (16 * (i & 1))) & 0xffffu);
        else
          f = mx_unpack_e2m1((c[u][i * CW / 8] >> (8 * (i & 3))) & 0xffu);
        o[i] = pack_bf16x2(f.x * s, f.y * s);
      }
      st_global_v8(x + p.row * K + k, o);
    }
  }
}

// s = bf16(x + residual); xn = bf16(s * (mean(s^2) + eps)^(-1/2) * gamma);
// codes, scales = MX(xn).  TPR threads hold a row, V vectors of 8 elements
// each (vector j*TPR + t, so that loads are whole lines), from the first load
// to the last store: every tensor is read once.  fp32 sum of squares in a fixed
// order (a thread's vectors, lanes by halving, warps in order).  sum may be x or
// residual: a thread writes what it alone has read.  FMT 0: no codes.
template <int FMT, int TPR, int V>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    add_rmsnorm_kernel(const uint4* x, const uint4* residual, const float4* __restrict__ gamma,
                       float eps, int T, int H, uint4* sum,
                       uint4* __restrict__ xn, uint8_t* __restrict__ codes,
                       uint32_t* __restrict__ scales) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int ROWS = BLOCK / TPR;  // rows of a block
  constexpr int WPR = TPR / 32;      // warps of a row
  __shared__ float part[BLOCK / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % TPR, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * ROWS + threadIdx.x / TPR;
  const bool live = row < T;
  const int nv = H / 8;
  uint4 v[V];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = j * TPR + t;
    v[j] = make_uint4(0, 0, 0, 0);
    if (live && c < nv) {
      v[j] = x[row * nv + c];
      if (residual) {
        const uint4 r = residual[row * nv + c];
        v[j].x = pack_bf16x2(bf16_lo(v[j].x) + bf16_lo(r.x), bf16_hi(v[j].x) + bf16_hi(r.x));
        v[j].y = pack_bf16x2(bf16_lo(v[j].y) + bf16_lo(r.y), bf16_hi(v[j].y) + bf16_hi(r.y));
        v[j].z = pack_bf16x2(bf16_lo(v[j].z) + bf16_lo(r.z), bf16_hi(v[j].z) + bf16_hi(r.z));
        v[j].w = pack_bf16x2(bf16_lo(v[j].w) + bf16_lo(r.w), bf16_hi(v[j].w) + bf16_hi(r.w));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ss = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), ss);
      ss = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), ss);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(FULL, ss, off);
  if constexpr (WPR > 1) {
    if (lane == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    const float* mine = part + (threadIdx.x / TPR) * WPR;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) ss += mine[i];
  }
  const float inv = 1.0f / sqrtf(ss / (float)H + eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = j * TPR + t;
    const bool in = live && c < nv;
    if (in && sum) sum[row * nv + c] = v[j];
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
    float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (gamma && c < nv) {
      const float4 a = gamma[2 * c], b = gamma[2 * c + 1];
      g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
      g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack_bf16x2(bf16_lo(w[i]) * inv * g[2 * i], bf16_hi(w[i]) * inv * g[2 * i + 1]);
    if (in && xn) xn[row * nv + c] = make_uint4(o[0], o[1], o[2], o[3]);
    if constexpr (FMT != 0) {
      // four lanes hold a block of 32, sixteen a word of scales
      uint32_t m = 0;
      if (in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = abs_max2(m, o[i]);
      }
      m = abs_max2(m, __shfl_xor_sync(FULL, m, 1));
      m = abs_max2(m, __shfl_xor_sync(FULL, m, 2));
      const uint32_t byte = mx_scale_byte<FMT>(amax_bits(m));
      uint32_t word = in ? byte << (8 * ((t >> 2) & 3)) : 0;
      word |= __shfl_xor_sync(FULL, word, 4);
      word |= __shfl_xor_sync(FULL, word, 8);
      if (in) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_lo(o[i]);
          f[2 * i + 1] = bf16_hi(o[i]);
        }
        uint32_t q[2];
        mx_encode<FMT>(f, byte, q);
        if constexpr (FMT == MOE_MXFP8)
          *reinterpret_cast<uint2*>(codes + row * H + 8 * c) = make_uint2(q[0], q[1]);
        else
          *reinterpret_cast<uint32_t*>(codes + (row * H + 8 * c) / 2) = q[0];
        if ((t & 15) == 0) scales[(long long)(c >> 4) * T + row] = word;
      }
    }
  }
}

template <int FMT, int TPR, int V>
cudaError_t launch_norm(const void* x, const void* residual, const float* gamma, float eps, int T,
                        int H, void* sum, void* xn, uint8_t* codes, uint32_t* scales,
                        cudaStream_t stream) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int ROWS = BLOCK / TPR;
  return launch_chained(add_rmsnorm_kernel<FMT, TPR, V>, dim3((T + ROWS - 1) / ROWS), dim3(BLOCK),
                        0, stream, static_cast<const uint4*>(x),
                        static_cast<const uint4*>(residual),
                        reinterpret_cast<const float4*>(gamma), eps, T, H,
                        static_cast<uint4*>(sum), static_cast<uint4*>(xn), codes, scales);
}

// Threads of a row: by its length alone (a row's bits do not depend on the batch),
// as many as give each thread one vector, then two and four.  H = 2048: 57 us at
// 19,412 rows with 256 threads of one vector (6.3 TB/s, 0.97 of the measured copy)
// against 65 with 64 threads of four, and 2.0 against 3.7 us for one row.
template <int FMT>
cudaError_t launch_norm_fmt(const void* x, const void* residual, const float* gamma, float eps,
                            int T, int H, void* sum, void* xn, uint8_t* codes, uint32_t* scales,
                            cudaStream_t s) {
  if (H <= 256)
    return launch_norm<FMT, 32, 1>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
  if (H <= 512)
    return launch_norm<FMT, 64, 1>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
  if (H <= 1024)
    return launch_norm<FMT, 128, 1>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
  if (H <= 2048)
    return launch_norm<FMT, 256, 1>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
  if (H <= 4096)
    return launch_norm<FMT, 512, 1>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
  if (H <= 8192)
    return launch_norm<FMT, 512, 2>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
  return launch_norm<FMT, 512, 4>(x, residual, gamma, eps, T, H, sum, xn, codes, scales, s);
}

// Words per lane: 4 where that still gives every SM 8 blocks, else 1.
template <typename F>
cudaError_t launch_by_words(long long total_rows, int K, F&& launch) {
  const unsigned rb = (unsigned)((total_rows + 31) / 32), words = mx_words(K);
  if ((long long)rb * ((words + 3) / 4) >= 8LL * num_sms())
    return launch(std::integral_constant<int, 4>(), dim3(rb, (words + 3) / 4));
  return launch(std::integral_constant<int, 1>(), dim3(rb, words));
}

}  // namespace

cudaError_t launch_mx_quantize(const void* x, int groups, int rows, int K, int fmt, uint8_t* codes,
                               uint8_t* scales, cudaStream_t stream) {
  const long long total = (long long)groups * rows;
  return launch_by_words(total, K, [&](auto u, dim3 grid) {
    constexpr int U = decltype(u)::value;
    auto k = fmt == MOE_MXFP8 ? mx_quantize_kernel<MOE_MXFP8, U> : mx_quantize_kernel<MOE_MXFP4, U>;
    return launch_chained(k, grid, dim3(256), 0, stream, static_cast<const __nv_bfloat16*>(x),
                          total, rows, K, mx_words(K), codes, reinterpret_cast<uint32_t*>(scales));
  });
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int groups, int rows,
                                 int K, int fmt, void* x, cudaStream_t stream) {
  const long long total = (long long)groups * rows;
  return launch_by_words(total, K, [&](auto u, dim3 grid) {
    constexpr int U = decltype(u)::value;
    auto k =
        fmt == MOE_MXFP8 ? mx_dequantize_kernel<MOE_MXFP8, U> : mx_dequantize_kernel<MOE_MXFP4, U>;
    return launch_chained(k, grid, dim3(256), 0, stream, codes,
                          reinterpret_cast<const uint32_t*>(scales), total, rows, K, mx_words(K),
                          static_cast<__nv_bfloat16*>(x));
  });
}

cudaError_t launch_add_rmsnorm(const void* x, const void* residual, const float* gamma, float eps,
                               int T, int H, int fmt, void* sum, void* xn, uint8_t* codes,
                               uint8_t* scales, cudaStream_t stream) {
  uint32_t* sw = reinterpret_cast<uint32_t*>(scales);
  switch (fmt) {
    case 0:
      return launch_norm_fmt<0>(x, residual, gamma, eps, T, H, sum, xn, codes, sw, stream);
    case MOE_MXFP8:
      return launch_norm_fmt<MOE_MXFP8>(x, residual, gamma, eps, T, H, sum, xn, codes, sw, stream);
    case MOE_MXFP4:
      return launch_norm_fmt<MOE_MXFP4>(x, residual, gamma, eps, T, H, sum, xn, codes, sw, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace rmoe

// 4-bit microscaled floating point: quantiser and its inverse, for 16-bit and FP32 tensors.
//
//   MXFP4  E2M1 codes, one UE8M0 byte per 32 values of a row: X = 2^e with e the smallest
//          integer >= -127 such that amax <= 6 * 2^e (nothing saturates), q = E2M1(v / X),
//          v / X exact;
//   NVFP4  E2M1 codes, one E4M3 byte S per 16 values, one FP32 tensor scale alpha:
//          S = E4M3(amax / (6 alpha)), q = E2M1(v / (S alpha)), every step an IEEE FP32
//          operation (the rule of beam_moe_quantize_nvfp4, whose codes these are).
// All roundings to nearest, ties to even.  A block that holds a NaN or an infinity gets a NaN
// scale (0xFF, 0x7F) and zero codes, so that it reads back, and multiplies, as NaN.
//
// Bound by memory: a 16-bit value costs 2 bytes to read and 0.53 or 0.56 to write.  The quantiser
// gives a thread a whole block (16 or 32 values), so that the block's scale is worked out once
// and without a shuffle; four lanes to a block of 8 values each, with its wider loads, spent the
// time on the scales instead (16384 x 5120 BF16: MXFP4 57, NVFP4 107 us).  The inverse gives a
// lane 8 values, whose store is then 16 bytes.
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/beam_moe.h"
#include "common.cuh"
#include "internal.h"
#include "overlap.h"

namespace beam {

namespace {

constexpr int kMxFp4 = BEAM_MOE_FP4_MX;
constexpr int kPieces = 4;      // pieces of 256 values that a warp has in flight
constexpr int kPieceValues = 256;

template <int TYPE>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
  if constexpr (TYPE == kTypeFp32) {
    const float4 a = __ldcg(static_cast<const float4*>(p)), b = __ldcg(static_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 q = __ldcg(static_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kTypeBf16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
}

// One 32-byte load from a 32-byte boundary.  (Not through the read-only path, here and below: the
// kernel may have started before the one that writes the memory ended.)
__device__ __forceinline__ void ld_global_v8(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// A block as it lies in memory, in 32-bit words (two 16-bit values or one FP32 value each).
template <int TYPE, int N>
struct RawBlock {
  static constexpr int kPer = TYPE == kTypeFp32 ? 1 : 2;
  static constexpr int kWords = N / kPer;
  uint32_t w[kWords];
  // wide: p lies on a 32-byte boundary
  __device__ __forceinline__ void load(const void* p, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8) ld_global_v8(static_cast<const uint32_t*>(p) + i, w + i);
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 q = __ldcg(static_cast<const uint4*>(p) + i);
      w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (TYPE == kTypeFp32) return __uint_as_float(w[i]);
    else if constexpr (TYPE == kTypeBf16) return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i / 2]);
      return (i & 1) ? __high2float(h) : __low2float(h);
    }
  }
  // The largest |v| as FP32 bits, which order like the values (NaN above infinity).  Of 16-bit
  // values, two maxima at a time on their own bits, which order likewise.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
    if constexpr (TYPE == kTypeFp32) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      m = max(m >> 16, m & 0xFFFFu);
      if constexpr (TYPE == kTypeBf16) return m << 16;
      else return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    }
  }
};

// A matrix cut into pieces, per_row to a row: blocks of 16 or 32 values, or 256 values of a row,
// the last such piece of a row shorter.  A matrix whose rows lie end to end in every array is one
// long row.  Rows are split from piece numbers by a multiplication; with magic =
// min(2^32 - 1, floor(2^32 / per_row)) the quotient is right or one too small.
struct Pieces {
  uint32_t total, per_row, magic;
};
__device__ __forceinline__ void split_piece(const Pieces& s, uint32_t p, uint32_t& row, uint32_t& rest) {
  row = __umulhi(p, s.magic);
  rest = p - row * s.per_row;
  if (rest >= s.per_row) {
    ++row;
    rest -= s.per_row;
  }
}
struct Piece {
  uint32_t row;
  int64_t col;  // the lane's first value
  bool in;      // the lane's 8 values lie in the row
};
__device__ __forceinline__ Piece piece_of(const Pieces& s, uint32_t p, int64_t cols, int lane) {
  Piece r;
  uint32_t rest;
  split_piece(s, p, r.row, rest);
  r.col = static_cast<int64_t>(rest) * kPieceValues + lane * 8;
  r.in = p < s.total && r.col < cols;
  return r;
}

// v / d rounded to nearest, r = 1 / d rounded to nearest.  Markstein's division (IBM J. Res. Dev.
// 34, 1990): with the reciprocal so rounded and q within a unit in the last place, q plus r times
// the remainder v - q d rounds to the quotient.  v r is within two units, the first step brings
// it within one, the second is exact; neither branches, and the remainder is one fused operation.
// Holds while nothing leaves the normal range (a quotient that does is a zero code all the same).
__device__ __forceinline__ float quotient(float v, float d, float r) {
  float q = __fmul_rn(v, r);
  q = __fmaf_rn(__fmaf_rn(-q, d, v), r, q);
  return __fmaf_rn(__fmaf_rn(-q, d, v), r, q);
}

template <int TYPE, int FORMAT>
__global__ void __launch_bounds__(256) quantize_fp4_kernel(const void* __restrict__ src, int64_t ld, Pieces blocks,
                                                           float alpha_param, const float* __restrict__ amax_dev,
                                                           uint8_t* __restrict__ codes, int64_t ldc,
                                                           uint8_t* __restrict__ sf, int64_t ldsf,
                                                           float* __restrict__ alpha_out, bool wide) {
  constexpr bool kMx = FORMAT == kMxFp4;
  constexpr int kSize = TYPE == kTypeFp32 ? 4 : 2;
  constexpr int N = kMx ? 32 : 16;
  constexpr int kAtOnce = N * kSize <= 64 ? 2 : 1;  // blocks a thread has in flight
  pdl_wait();
  pdl_trigger();
  const uint32_t threads = gridDim.x * 256u;
  float alpha = 0.0f, six_alpha = 0.0f;
  if (!kMx) {
    alpha = amax_dev ? __fdiv_rn(__ldcg(amax_dev), 2688.0f) : alpha_param;
    six_alpha = __fmul_rn(6.0f, alpha);
    if (alpha_out && blockIdx.x == 0 && threadIdx.x == 0) *alpha_out = alpha;
  }
  for (uint32_t q0 = blockIdx.x * 256u + threadIdx.x; q0 < blocks.total; q0 += threads * kAtOnce) {
    RawBlock<TYPE, N> raw[kAtOnce];
    uint32_t row[kAtOnce], col[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t q = q0 + u * threads;
      split_piece(blocks, q, row[u], col[u]);
      if (q < blocks.total)
        raw[u].load(static_cast<const uint8_t*>(src) + (row[u] * ld + static_cast<int64_t>(col[u]) * N) * kSize,
                    wide);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (q0 + u * threads >= blocks.total) break;
      const uint32_t m = raw[u].amax();
      const bool finite = m < 0x7F800000u;
      uint32_t scale, word[N / 8];
#pragma unroll
      for (int i = 0; i < N / 8; ++i) word[i] = 0;
      if constexpr (kMx) {
        // amax = f * 2^E, f in [1, 2): 6 = 1.5 * 2^2, so e = E - 2 where f <= 1.5, else E - 1
        int e = static_cast<int>(m >> 23) - 127 - 2 + ((m & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        e = max(e, -127);
        scale = finite ? static_cast<uint32_t>(e + 127) : 0xFFu;
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e in [-127, 126]
        if (finite) {
#pragma unroll
          for (int i = 0; i < N / 2; ++i)
            word[i / 4] |= cvt_e2m1x2(__fmul_rn(raw[u].value(2 * i), inv), __fmul_rn(raw[u].value(2 * i + 1), inv))
                           << (8 * (i & 3));
        }
      } else {
        scale = alpha > 0.0f ? cvt_e4m3(__fdiv_rn(__uint_as_float(m), six_alpha)) : 0u;
        if (!finite) scale = 0x7Fu;
        if (finite && scale != 0) {
          const float d = __fmul_rn(e4m3_value(scale), alpha);
          const float r = __frcp_rn(d);
          // no step leaves FP32's normal range (a saturated block scale makes large quotients)
          if (d >= 0x1p-100f && d <= 0x1p100f && __uint_as_float(m) <= d * 0x1p20f) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
              word[i / 4] |= cvt_e2m1x2(quotient(raw[u].value(2 * i), d, r), quotient(raw[u].value(2 * i + 1), d, r))
                             << (8 * (i & 3));
          } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
              word[i / 4] |= cvt_e2m1x2(__fdiv_rn(raw[u].value(2 * i), d), __fdiv_rn(raw[u].value(2 * i + 1), d))
                             << (8 * (i & 3));
          }
        }
      }
      uint8_t* c = codes + row[u] * ldc + static_cast<int64_t>(col[u]) * (N / 2);
      if constexpr (kMx)
        *reinterpret_cast<uint4*>(c) = make_uint4(word[0], word[1], word[2], word[3]);
      else
        *reinterpret_cast<uint2*>(c) = make_uint2(word[0], word[1]);
      sf[row[u] * ldsf + col[u]] = static_cast<uint8_t>(scale);
    }
  }
}

// The largest finite |v|, as FP32 bits.
template <int TYPE>
__global__ void __launch_bounds__(256) amax_finite_kernel(const void* __restrict__ src, int64_t ld, Pieces pieces,
                                                          int64_t cols, unsigned int* __restrict__ out) {
  constexpr int kSize = TYPE == kTypeFp32 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * 8u;
  uint32_t m = 0;
  for (uint32_t p0 = blockIdx.x * 8u + (threadIdx.x >> 5); p0 < pieces.total; p0 += warps * kPieces) {
    float v[kPieces][8];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const Piece at = piece_of(pieces, p0 + u * warps, cols, lane);
      if (at.in)
        load8<TYPE>(static_cast<const uint8_t*>(src) + (at.row * ld + at.col) * kSize, v[u]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[u][i]) & 0x7FFFFFFFu;
        if (b < 0x7F800000u) m = max(m, b);
      }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  __shared__ uint32_t wm[8];
  if (lane == 0) wm[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) m = max(m, wm[i]);
    if (m) atomicMax(out, m);
  }
}

// Two E2M1 codes (a byte) -> two FP32 values, exact.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A thread turns 32 bytes' worth of values: 16 of 16 bits or 8 of 32.
template <int OUT>
constexpr int kOutValues = OUT == kTypeFp32 ? 8 : 16;

template <int FORMAT, int OUT>
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                             const uint8_t* __restrict__ sf, int64_t ldsf,
                                                             const float* __restrict__ alpha_dev, Pieces pieces,
                                                             void* __restrict__ out, int64_t ldo, bool wide) {
  constexpr bool kMx = FORMAT == kMxFp4;
  constexpr int V = kOutValues<OUT>, kAtOnce = 4;
  pdl_wait();
  pdl_trigger();
  const uint32_t threads = gridDim.x * 256u;
  const float alpha = !kMx && alpha_dev ? __ldcg(alpha_dev) : 1.0f;
  for (uint32_t q0 = blockIdx.x * 256u + threadIdx.x; q0 < pieces.total; q0 += threads * kAtOnce) {
    uint32_t word[kAtOnce][V / 8], scale[kAtOnce], row[kAtOnce], part[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t q = q0 + u * threads;
      split_piece(pieces, q, row[u], part[u]);
      if (q < pieces.total) {
        const uint8_t* c = codes + row[u] * ldc + static_cast<int64_t>(part[u]) * (V / 2);
        if constexpr (V == 16) {
          const uint2 w = __ldcg(reinterpret_cast<const uint2*>(c));
          word[u][0] = w.x;
          word[u][1] = w.y;
        } else {
          word[u][0] = __ldcg(reinterpret_cast<const uint32_t*>(c));
        }
        scale[u] = __ldcg(sf + row[u] * ldsf + static_cast<int64_t>(part[u]) * V / (kMx ? 32 : 16));
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (q0 + u * threads >= pieces.total) break;
      float s;
      if constexpr (kMx) {  // 2^(scale - 127); 0 is the subnormal 2^-127
        s = scale[u] == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(scale[u] << 23);
        if (scale[u] == 0xFFu) s = __uint_as_float(0x7FC00000u);
      } else {
        s = (scale[u] & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_value(scale[u] & 0x7Fu);
      }
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 q = e2m1x2_values((word[u][i / 4] >> (8 * (i & 3))) & 0xFFu);
        // code times block scale is exact; the tensor scale is one FP32 rounding
        const float x = kMx ? __fmul_rn(q.x, s) : __fmul_rn(__fmul_rn(q.x, s), alpha);
        const float y = kMx ? __fmul_rn(q.y, s) : __fmul_rn(__fmul_rn(q.y, s), alpha);
        if constexpr (OUT == kTypeFp32) {
          w[2 * i] = __float_as_uint(x);
          w[2 * i + 1] = __float_as_uint(y);
        } else if constexpr (OUT == kTypeBf16) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
          const __half2 b = __floats2half2_rn(x, y);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      uint8_t* p = static_cast<uint8_t*>(out) +
                   (row[u] * ldo + static_cast<int64_t>(part[u]) * V) * (OUT == kTypeFp32 ? 4 : 2);
      if (wide) {
        st_global_v8(p, w);
      } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

// Up to `per_sm` CTAs of 256 threads an SM, each taking `each` pieces at a time.
unsigned grid_of(const Pieces& p, int each, int per_sm = 8) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((int64_t{p.total} + each - 1) / each, 148 * per_sm)));
}
// One launch's share of a matrix: at most kMaxPieces pieces, so that their numbers (and the steps
// of a loop past the last one) fit 32 bits.
constexpr int64_t kMaxPieces = int64_t{1} << 30;
Pieces pieces_of(int64_t rows, int64_t cols, int values) {
  const int64_t per_row = (cols + values - 1) / values;
  return Pieces{static_cast<uint32_t>(rows * per_row), static_cast<uint32_t>(per_row),
                static_cast<uint32_t>(std::min<int64_t>((int64_t{1} << 32) / per_row, 0xFFFFFFFFll))};
}
// Calls f(first row, rows, columns) for shares of the matrix, one long row where `flat`.
template <class F>
cudaError_t for_shares(int64_t rows, int64_t cols, int values, bool flat, F f) {
  if (flat && (rows * cols + values - 1) / values <= kMaxPieces) return f(int64_t{0}, int64_t{1}, rows * cols);
  const int64_t most = std::max<int64_t>(1, kMaxPieces / ((cols + values - 1) / values));
  for (int64_t r = 0; r < rows; r += most) {
    const cudaError_t e = f(r, std::min(most, rows - r), cols);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int TYPE>
cudaError_t launch_quantize(int format, const void* src, int64_t ld, int64_t rows, int cols, float alpha,
                            const float* amax_dev, uint8_t* codes, int64_t ldc, uint8_t* sf, int64_t ldsf,
                            float* alpha_out, cudaStream_t s) {
  auto k = format == kMxFp4 ? quantize_fp4_kernel<TYPE, BEAM_MOE_FP4_MX> : quantize_fp4_kernel<TYPE, BEAM_MOE_FP4_NV>;
  const bool flat = ld == cols && ldc == cols / 2 && ldsf == cols / (format == kMxFp4 ? 32 : 16);
  const int values = format == kMxFp4 ? 32 : 16;
  const bool wide = aligned_to(src, 32) && (rows == 1 || ld * (TYPE == kTypeFp32 ? 4 : 2) % 32 == 0);
  return for_shares(rows, cols, values, flat, [&](int64_t r, int64_t n, int64_t c) {
    const Pieces p = pieces_of(n, c, values);
    return launch_pdl(k, dim3(grid_of(p, 256)), dim3(256), 0, s,
                      static_cast<const uint8_t*>(src) + r * ld * (TYPE == kTypeFp32 ? 4 : 2), ld, p, alpha,
                      amax_dev, codes + r * ldc, ldc, sf + r * ldsf, ldsf, alpha_out, wide);
  });
}

template <int TYPE>
cudaError_t launch_amax_finite(const void* src, int64_t ld, int64_t rows, int cols, float* out, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(out, 0, sizeof(float), s);
  if (e != cudaSuccess) return e;
  return for_shares(rows, cols, kPieceValues, ld == cols, [&](int64_t r, int64_t n, int64_t c) {
    const Pieces p = pieces_of(n, c, kPieceValues);
    amax_finite_kernel<TYPE><<<grid_of(p, 8), 256, 0, s>>>(
        static_cast<const uint8_t*>(src) + r * ld * (TYPE == kTypeFp32 ? 4 : 2), ld, p, c,
        reinterpret_cast<unsigned int*>(out));
    return cudaGetLastError();
  });
}

template <int FORMAT>
cudaError_t launch_dequantize(int out_type, const uint8_t* codes, int64_t ldc, const uint8_t* sf, int64_t ldsf,
                              const float* alpha, int64_t rows, int cols, void* out, int64_t ldo, cudaStream_t s) {
  auto k = out_type == kTypeBf16   ? dequantize_fp4_kernel<FORMAT, kTypeBf16>
           : out_type == kTypeFp16 ? dequantize_fp4_kernel<FORMAT, kTypeFp16>
                                   : dequantize_fp4_kernel<FORMAT, kTypeFp32>;
  const bool flat = ldo == cols && ldc == cols / 2 && ldsf == cols / (FORMAT == kMxFp4 ? 32 : 16);
  const int values = out_type == kTypeFp32 ? kOutValues<kTypeFp32> : kOutValues<kTypeBf16>;
  const bool wide = aligned_to(out, 32) && (rows == 1 || ldo * (out_type == kTypeFp32 ? 4 : 2) % 32 == 0);
  return for_shares(rows, cols, values, flat, [&](int64_t r, int64_t n, int64_t c) {
    const Pieces p = pieces_of(n, c, values);
    return launch_pdl(k, dim3(grid_of(p, 256)), dim3(256), 0, s, codes + r * ldc, ldc, sf + r * ldsf, ldsf, alpha, p,
                      static_cast<void*>(static_cast<uint8_t*>(out) + r * ldo * (out_type == kTypeFp32 ? 4 : 2)), ldo,
                      wide);
  });
}

beam_moe_status check_fp4(int32_t format, int64_t rows, int32_t cols, int32_t type) {
  if (rows < 0 || cols < 0 || (format != BEAM_MOE_FP4_MX && format != BEAM_MOE_FP4_NV)) return BEAM_MOE_ERR_INVALID_ARG;
  if (type != BEAM_MOE_BF16 && type != BEAM_MOE_FP16 && type != BEAM_MOE_FP32) return BEAM_MOE_ERR_INVALID_ARG;
  // 2^46 values: products of rows and columns stay far inside 64 bits
  if (cols % 32 != 0 || rows > (int64_t{1} << 46) / std::max(cols, 32)) return BEAM_MOE_ERR_UNSUPPORTED;
  return BEAM_MOE_OK;
}
int scale_bytes(int32_t format, int32_t cols) { return cols / (format == BEAM_MOE_FP4_MX ? 32 : 16); }

}  // namespace

}  // namespace beam

using namespace beam;

extern "C" {

beam_moe_status beam_moe_quantize_fp4(int32_t format, const void* src, int32_t src_type, int64_t ld, int64_t rows,
                                      int32_t cols, float alpha, uint8_t* codes, int64_t ldc, uint8_t* sf,
                                      int64_t ldsf, float* alpha_out, void* stream) {
  const beam_moe_status st = check_fp4(format, rows, cols, src_type);
  if (st != BEAM_MOE_OK) return st;
  if (rows == 0 || cols == 0) return BEAM_MOE_OK;
  const int size = src_type == BEAM_MOE_FP32 ? 4 : 2;
  if (!src || !codes || !sf || !aligned_to(src, 16) || !aligned_to(codes, 16) || !aligned_to(sf, 16))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (ld < cols || ld * size % 16 != 0 || ldc < cols / 2 || ldc % 16 != 0 || ldsf < scale_bytes(format, cols) ||
      ldsf % 16 != 0)
    return BEAM_MOE_ERR_INVALID_ARG;
  const bool nv = format == BEAM_MOE_FP4_NV;
  const bool given = alpha > 0.0f && alpha <= 3.4028235e38f;
  if (nv && !given && (!(alpha <= 0.0f) || !alpha_out)) return BEAM_MOE_ERR_INVALID_ARG;  // infinite, NaN
  if (nv && alpha_out && !aligned_to(alpha_out, 4)) return BEAM_MOE_ERR_INVALID_ARG;
  const Span in{src, rows, static_cast<int64_t>(cols) * size, ld * size}, out_codes{codes, rows, cols / 2, ldc},
      out_sf{sf, rows, scale_bytes(format, cols), ldsf}, out_alpha{nv ? alpha_out : nullptr, 1, 4, 4};
  if (overlaps_any(in, {out_codes, out_sf, out_alpha}) || overlaps_any(out_codes, {out_sf, out_alpha}) ||
      overlap(out_sf, out_alpha))
    return BEAM_MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const float* amax = nullptr;
  if (nv && !given) {
    // alpha_out first holds the largest value, then the scale
    auto find = src_type == kTypeBf16   ? launch_amax_finite<kTypeBf16>
                : src_type == kTypeFp16 ? launch_amax_finite<kTypeFp16>
                                        : launch_amax_finite<kTypeFp32>;
    if (find(src, ld, rows, cols, alpha_out, s) != cudaSuccess) return BEAM_MOE_ERR_CUDA;
    amax = alpha_out;
  }
  auto run = src_type == kTypeBf16   ? launch_quantize<kTypeBf16>
             : src_type == kTypeFp16 ? launch_quantize<kTypeFp16>
                                     : launch_quantize<kTypeFp32>;
  // a given scale is written by the quantiser; one that it reads as the amax, only after it
  if (run(format, src, ld, rows, cols, alpha, amax, codes, ldc, sf, ldsf, amax ? nullptr : alpha_out, s) != cudaSuccess)
    return BEAM_MOE_ERR_CUDA;
  if (amax) return launch_status(launch_amax_to_alpha(alpha_out, s));
  return BEAM_MOE_OK;
}

beam_moe_status beam_moe_dequantize_fp4(int32_t format, const uint8_t* codes, int64_t ldc, const uint8_t* sf,
                                        int64_t ldsf, const float* alpha, int64_t rows, int32_t cols, void* out,
                                        int32_t out_type, int64_t ldo, void* stream) {
  const beam_moe_status st = check_fp4(format, rows, cols, out_type);
  if (st != BEAM_MOE_OK) return st;
  if (rows == 0 || cols == 0) return BEAM_MOE_OK;
  const int size = out_type == BEAM_MOE_FP32 ? 4 : 2;
  if (!codes || !sf || !out || !aligned_to(codes, 16) || !aligned_to(out, 16) || (alpha && !aligned_to(alpha, 4)))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (ldo < cols || ldo * size % 16 != 0 || ldc < cols / 2 || ldc % 16 != 0 || ldsf < scale_bytes(format, cols))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (overlaps_any({out, rows, static_cast<int64_t>(cols) * size, ldo * size},
                   {{codes, rows, cols / 2, ldc}, {sf, rows, scale_bytes(format, cols), ldsf},
                    {format == BEAM_MOE_FP4_NV ? alpha : nullptr, 1, 4, 4}}))
    return BEAM_MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = format == BEAM_MOE_FP4_MX ? launch_dequantize<BEAM_MOE_FP4_MX> : launch_dequantize<BEAM_MOE_FP4_NV>;
  return launch_status(run(out_type, codes, ldc, sf, ldsf, alpha, rows, cols, out, ldo, s));
}

}  // extern "C"

// RMSNorm with the residual's addition, in front of the MoE layer.
//
//   s = x + residual (fp32, rounded to the residual stream's type)
//   y = s * (mean(s^2) + eps)^-1/2 * gamma
// with y in bf16, or quantised to E4M3 with one fp32 scale per 128 columns
// (c = max(max|y|, 2^-100) / 448, q = e4m3(y / c)), or both.
//
// One block per row. Every thread keeps 16 (or 32) of the row's elements in
// registers between the sum of squares and the output, so the row is read
// once; 16 elements are one 32-byte bf16 vector, and 8 neighbouring threads
// hold one quantisation block of 128, whose maximum stays in the warp. The
// sum of squares is fp32: 16 terms per thread, then a tree.
//
// Memory bound: x, the residual and the outputs each cross once. 8192 x 2880
// with a bf16 residual takes 32.5 us (5.8 TB/s, 88% of the measured copy rate),
// 16384 x 2880 with E4M3 output 55.7 us (6.0 TB/s, 91%). A persistent grid whose
// blocks load the next row while they finish one was no faster (33.1 and 55.4 us
// at 1536 threads an SM, 41.3 and 72.0 at 1024): with 34 registers a thread ten
// blocks share an SM and overlap each other.
#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int kVec = 16;              // elements per vector
constexpr int kMaxThreads = 512;
constexpr float kAmaxMin = 7.888609052210118e-31f;  // 2^-100: keeps 448 / amax finite
constexpr float kE4m3Max = 448.0f;

struct NormParams {
  int D, vecs;  // row length, vectors per row
  int64_t ldx;
  float eps;
  const uint16_t* x;
  const void* residual;
  const uint16_t* gamma;
  void* res_out;
  uint16_t* y;
  uint8_t* q;
  float* q_scale;
};

__device__ __forceinline__ void unpack16(const uint32_t (&w)[8], float (&f)[kVec]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void pack16(const float (&f)[kVec], uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
}

// y / c for two y from inv, about 1 / c: first quotients and one Newton step with
// their remainders, which the FMA gives exactly. A quotient of few bits, such as
// one half-way between two E4M3 values, comes out exactly; y * inv alone can lie
// past it, which is a whole step of E4M3. (16384 x 2880: 55.3 us without the step,
// 55.5 with it, 57.3 one y at a time, 64.2 with fp32 divisions.)
__device__ __forceinline__ float2 quotients(float y0, float y1, float c, float inv) {
  float2 q;
  asm("{\n\t.reg .b64 y, d, i, f, r;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "mov.b64 d, {%4, %4};\n\t"
      "mov.b64 i, {%5, %5};\n\t"
      "mul.rn.f32x2 f, y, i;\n\t"
      "fma.rn.f32x2 r, f, d, y;\n\t"
      "fma.rn.f32x2 f, r, i, f;\n\t"
      "mov.b64 {%0, %1}, f;\n\t}"
      : "=f"(q.x), "=f"(q.y)
      : "f"(y0), "f"(y1), "f"(-c), "f"(inv));
  return q;
}

// kRes: 0 no residual, 1 bf16, 2 fp32. kN: vectors per thread.
template <int kRes, int kN>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_kernel(const NormParams p) {
  using namespace sm100;
  __shared__ float part[kMaxThreads / 32];
  const int64_t row = blockIdx.x;
  float v[kN][kVec];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int vec = threadIdx.x + j * blockDim.x;
    if (vec < p.vecs) {
      uint32_t w[8];
      // plain loads: residual and res_out may be the same buffer
      ld_global_v8u(p.x + row * p.ldx + vec * kVec, w);
      unpack16(w, v[j]);
      if (kRes == 1) {
        uint32_t r[8];
        ld_global_plain_v8u(static_cast<const uint16_t*>(p.residual) + row * p.D + vec * kVec, r);
        float f[kVec];
        unpack16(r, f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] += f[i];
        pack16(v[j], r);
        if (p.res_out) st_global_v8u(static_cast<uint16_t*>(p.res_out) + row * p.D + vec * kVec, r);
        unpack16(r, v[j]);  // the norm is that of the stored stream
      } else if (kRes == 2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[8];
          ld_global_plain_v8u(static_cast<const float*>(p.residual) + row * p.D + vec * kVec + 8 * half, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[j][8 * half + i] += __uint_as_float(r[i]);
            r[i] = __float_as_uint(v[j][8 * half + i]);
          }
          if (p.res_out) st_global_v8u(static_cast<float*>(p.res_out) + row * p.D + vec * kVec + 8 * half, r);
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum = fmaf(v[j][i], v[j][i], sum);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
  __syncthreads();
  float total = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) total += part[i];
  const float rstd = rsqrtf(total / static_cast<float>(p.D) + p.eps);

  const int qblocks = (p.D + 127) / 128;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int vec = threadIdx.x + j * blockDim.x;
    const bool on = vec < p.vecs;
    float amax = 0.0f;
    if (on) {
      uint32_t g[8];
      ld_global_v8u(p.gamma + vec * kVec, g);
      float f[kVec];
      unpack16(g, f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[j][i] = v[j][i] * rstd * f[i];
        amax = max_nan(amax, fabsf(v[j][i]));
      }
      if (p.y) {
        uint32_t w[8];
        pack16(v[j], w);
        st_global_v8u(p.y + row * p.D + vec * kVec, w);
      }
    }
    if (p.q) {  // (uniform: every lane takes part in the shuffles)
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      if (on) {
        amax = max_nan(amax, kAmaxMin);
        const float c = amax / kE4m3Max, inv = kE4m3Max / amax;
        const float back = isinf(c) ? 0.0f : c;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo =
              __nv_cvt_float2_to_fp8x2(quotients(v[j][4 * i], v[j][4 * i + 1], back, inv), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(quotients(v[j][4 * i + 2], v[j][4 * i + 3], back, inv),
                                                       __NV_SATFINITE, __NV_E4M3);
          w[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4*>(p.q + row * p.D + vec * kVec) = make_uint4(w[0], w[1], w[2], w[3]);
        if (vec % 8 == 0) p.q_scale[row * qblocks + vec / 8] = c;
      }
    }
  }
}

template <int kN>
void launch(const NormParams& p, int T, int res, int threads, cudaStream_t s) {
  if (res == 0)
    rmsnorm_kernel<0, kN><<<T, threads, 0, s>>>(p);
  else if (res == 1)
    rmsnorm_kernel<1, kN><<<T, threads, 0, s>>>(p);
  else
    rmsnorm_kernel<2, kN><<<T, threads, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_rmsnorm(const moe_norm_t& n, const uint16_t* x, const void* residual, const uint16_t* gamma,
                           void* res_out, uint16_t* y, uint8_t* q, float* q_scale, cudaStream_t s) {
  NormParams p{};
  p.D = n.D;
  p.vecs = n.D / kVec;
  p.ldx = n.ldx;
  p.eps = n.eps;
  p.x = x;
  p.residual = residual;
  p.gamma = gamma;
  p.res_out = res_out;
  p.y = y;
  p.q = q;
  p.q_scale = q_scale;
  const int res = !residual ? 0 : n.res_type == MOE_T_BF16 ? 1 : 2;
  // one vector per thread while a row fits a block, two beyond
  if (p.vecs <= kMaxThreads)
    launch<1>(p, n.T, res, (p.vecs + 31) / 32 * 32, s);
  else
    launch<2>(p, n.T, res, ((p.vecs + 1) / 2 + 31) / 32 * 32, s);
  return cudaGetLastError();
}

}  // namespace moe

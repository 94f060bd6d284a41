// block_norm.cu -- the norms before and after a block with its gate and residual.
//
// Per row of d values:
//     u = post ? x / sqrt(mean(x^2) + eps_post) * w_post : x
//     r = residual + alpha * gate * u            -> residual_out (its type)
//     y = r / sqrt(mean(r^2) + eps_pre) * w_pre  -> bf16
// in fp32; y is made from the unrounded r.  Memory-bound: x, the residual and a gate of
// every row are read once, the new residual and y written once.
//
// One CTA per row; thread t holds the 8-value vectors t, t + blockDim, ... of the row in
// registers, so the row is read once although both norms need all of it.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_common.cuh"
#include "gdr_host.h"

namespace gdr {
namespace {

constexpr int kVec = 4;   // 8-value vectors a thread can hold

__device__ __forceinline__ float block_sum(float v, float *s_part) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  __syncthreads();   // the last sum's reads are done
  if ((threadIdx.x & 31) == 0) s_part[warp] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < warps; ++w) t += s_part[w];
  return t;
}

__device__ __forceinline__ void load_f8(const float *p, float *f) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__global__ void block_norm_kernel(const BlockNormParams p) {
  __shared__ float s_part[32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = blockIdx.x;
  const int nv = p.d >> 3;
  float r[kVec][8];
  const uint16_t *x = p.x + row * p.x_stride;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nv) {
      unpack8(*reinterpret_cast<const uint4 *>(x + 8 * c), r[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += r[i][e] * r[i][e];
    }
  }
  float f = p.alpha;
  if (p.post) f *= 1.0f / sqrtf(block_sum(ss, s_part) / static_cast<float>(p.d) + p.eps_post);
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nv) {
      float m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] *= f;
      if (p.post && p.w_post) {
        load_f8(p.w_post + 8 * c, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] *= m[e];
      }
      if (p.gate) {
        unpack8(*reinterpret_cast<const uint4 *>(p.gate + row * p.gate_stride + 8 * c), m);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] *= m[e];
      }
      if (p.res) {
        if (p.res_fp32) load_f8(static_cast<const float *>(p.res) + row * p.res_stride + 8 * c, m);
        else unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.res) + row * p.res_stride + 8 * c), m);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] += m[e];
      }
      if (p.out) {
        if (p.res_fp32) {
          float *w = static_cast<float *>(p.out) + row * p.out_stride + 8 * c;
          *reinterpret_cast<float4 *>(w) = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
          *reinterpret_cast<float4 *>(w + 4) = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        } else {
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + row * p.out_stride + 8 * c) = pack8x2(r[i]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += r[i][e] * r[i][e];
    }
  }
  if (!p.y) return;
  const float inv = 1.0f / sqrtf(block_sum(ss, s_part) / static_cast<float>(p.d) + p.eps_pre);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nv) {
      float m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] *= inv;
      if (p.w_pre) {
        load_f8(p.w_pre + 8 * c, m);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] *= m[e];
      }
      *reinterpret_cast<uint4 *>(p.y + row * p.y_stride + 8 * c) = pack8x2(r[i]);
    }
  }
}

}  // namespace

int launch_block_norm(const BlockNormParams &p, int64_t rows, cudaStream_t s) {
  if (rows > 0x7FFFFFFF) return GDR_ERR_SHAPE;
  const int nv = p.d >> 3;
  const int threads = ((nv + kVec - 1) / kVec + 31) / 32 * 32;
  return launch_status(launch_pdl(block_norm_kernel, dim3(static_cast<unsigned>(rows)), dim3(threads), 0, s, 1, p),
                       "block norm: kernel launch");
}

}  // namespace gdr

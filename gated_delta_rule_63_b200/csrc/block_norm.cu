// block_norm.cu -- the norms before and after a block with its gate and residual.
//
// Per row of d values:
//     u = post ? x / sqrt(mean(x^2) + eps_post) * w_post : x
//     r = residual + alpha * gate * u            -> residual_out (its type)
//     y = r / sqrt(mean(r^2) + eps_pre) * w_pre  -> bf16
// in fp32; y is made from the unrounded r.  Memory-bound: x, the residual and a gate of
// every row are read once, the new residual and y written once.
//
// A row is held in registers, so it is read once although both norms need all of it, and all
// its loads are issued before the first sum (loads behind the sums: 4096 rows of 5120 took 38.6
// instead of 26.9 us).  Up to 512 values a warp holds a row, four rows a CTA, and sums with
// shuffles alone (16 384 rows of 512: 9.9 us, 17.5 us with a CTA a row); above, a CTA of up to
// 512 threads does (64 rows of 1024: 2.1 us, 2.7 us with a warp a row; 16 384 rows 20.4 and
// 20.6 us), 16 values a thread up to 8192 (4096 rows of 8192: 41.4 us, 49.1 us with 8 values
// a thread; of 5120 26.9, with 8 values 29.8, with 32 27.2 us), 32 up to 16384 (2048 rows of 16 384
// with everything and an fp32 residual: 94 us, 130 us with 64 values; residual and norm alone 45 and
// 49 us; of 8192 33.6 million values so: 16 values 82 us, 32 86 us), 64 above, the only form whose 512
// threads reach 32 768.  That one needs more registers than a thread has (up to 228 bytes go to local
// memory and come back) and takes 56 to 69 us for 33.6 million values, with everything 138 to 183 us.
// Residual + norm of 4096 x 5120 bf16 in 28 us moves 168 MB, 6.0 TB/s: 91% of a copy's rate; with the
// residual in fp32 40.8 us, 252 MB: 94%, with both norms and a row's gate 52 us, 294 MB: 86%.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_common.cuh"
#include "gdr_host.h"

namespace gdr {
namespace {

constexpr int kWarpRows = 4;   // rows (warps) of a CTA where a warp holds a row

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum over the warp (kWarp) or the CTA; `part` is 32 floats of shared memory of this sum alone.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float *part) {
  v = warp_sum(v);
  if (kWarp) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? part[lane] : 0.0f);
}

__device__ __forceinline__ void mul8(float *r, const float *m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] *= m[e];
}
__device__ __forceinline__ void get8(const float4 *p, float *f) {
  const float4 a = __ldg(p), b = __ldg(p + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ float sum_sq8(const float *f) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += f[e] * f[e];
  return s;
}

// Thread t of a row's `width` threads holds the 8-value vectors t, t + width, ... (NV of them).
template <int NV, bool kWarp, bool kPost, bool kWide>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : 512)
block_norm_kernel(const __grid_constant__ BlockNormParams p) {
  __shared__ float s_part[2][32];
  const int width = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const int nv = p.d >> 3;
  grid_dep_wait();
  grid_dep_launch();
  if (kWarp && row >= p.rows) return;

  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 x[NV], gate[NV], res[NV * (kWide ? 2 : 1)];
  const uint4 *px = reinterpret_cast<const uint4 *>(p.x + row * p.x_stride);
  const uint4 *pg = reinterpret_cast<const uint4 *>(p.gate + row * p.gate_stride);
  const uint4 *pr = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.res) + row * p.res_stride * (kWide ? 4 : 2));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * width;
    const bool in = c < nv;
    x[i] = in ? px[c] : zero;
    if (p.res) {
      if (kWide) {
        res[2 * i] = in ? pr[2 * c] : zero;
        res[2 * i + 1] = in ? pr[2 * c + 1] : zero;
      } else {
        res[i] = in ? pr[c] : zero;
      }
    }
    if (p.gate) gate[i] = in ? pg[c] : zero;
  }

  float r[NV][8];
  float f = p.alpha;
  if (kPost) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack8(x[i], r[i]);
      ss += sum_sq8(r[i]);
    }
    f *= 1.0f / sqrtf(row_sum<kWarp>(ss, s_part[0]) / static_cast<float>(p.d) + p.eps_post);
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * width;
    if (c >= nv) continue;
    float m[8];
    if (!kPost) unpack8(x[i], r[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] *= f;
    if (kPost && p.w_post) {
      get8(reinterpret_cast<const float4 *>(p.w_post) + 2 * c, m);
      mul8(r[i], m);
    }
    if (p.gate) {
      unpack8(gate[i], m);
      mul8(r[i], m);
    }
    if (p.res) {
      if (kWide) {
        const uint4 a = res[2 * i], b = res[2 * i + 1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = __uint_as_float(w[e]);
      } else {
        unpack8(res[i], m);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] += m[e];
    }
    ss += sum_sq8(r[i]);
    if (p.out) {
      uint8_t *out = static_cast<uint8_t *>(p.out) + (row * p.out_stride + 8 * c) * (kWide ? 4 : 2);
      if (kWide) {
        reinterpret_cast<float4 *>(out)[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
        reinterpret_cast<float4 *>(out)[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
      } else {
        *reinterpret_cast<uint4 *>(out) = pack8x2(r[i]);
      }
    }
  }
  if (!p.y) return;
  const float inv = 1.0f / sqrtf(row_sum<kWarp>(ss, s_part[1]) / static_cast<float>(p.d) + p.eps_pre);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * width;
    if (c >= nv) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] *= inv;
    if (p.w_pre) {
      float m[8];
      get8(reinterpret_cast<const float4 *>(p.w_pre) + 2 * c, m);
      mul8(r[i], m);
    }
    *reinterpret_cast<uint4 *>(p.y + row * p.y_stride + 8 * c) = pack8x2(r[i]);
  }
}

template <int NV, bool kWarp>
cudaError_t launch(const BlockNormParams &p, cudaStream_t s) {
  const int per_cta = kWarp ? kWarpRows : 1;
  const dim3 grid(static_cast<unsigned>((p.rows + per_cta - 1) / per_cta));
  const dim3 block(kWarp ? 32 * kWarpRows : ((p.d >> 3) + NV * 32 - 1) / (NV * 32) * 32);
  if (p.post)
    return p.res_fp32 ? launch_pdl(block_norm_kernel<NV, kWarp, true, true>, grid, block, 0, s, 1, p)
                      : launch_pdl(block_norm_kernel<NV, kWarp, true, false>, grid, block, 0, s, 1, p);
  return p.res_fp32 ? launch_pdl(block_norm_kernel<NV, kWarp, false, true>, grid, block, 0, s, 1, p)
                    : launch_pdl(block_norm_kernel<NV, kWarp, false, false>, grid, block, 0, s, 1, p);
}

}  // namespace

int launch_block_norm(const BlockNormParams &p, cudaStream_t s) {
  if (p.rows > 0x7FFFFFFF) return GDR_ERR_SHAPE;
  const int d = p.d;
  const cudaError_t e = d <= 256     ? launch<1, true>(p, s)
                        : d <= 512   ? launch<2, true>(p, s)
                        : d <= 8192  ? launch<2, false>(p, s)
                        : d <= 16384 ? launch<4, false>(p, s)
                                     : launch<8, false>(p, s);
  return launch_status(e, "block norm: kernel launch");
}

}  // namespace gdr

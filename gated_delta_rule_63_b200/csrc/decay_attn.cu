// decay_attn.cu -- decayed linear attention over packed sequences.
//
// Per sequence and value head, with l = exp(log_decay[h]) and H the [dk][dv] fp32 state:
//     H_t = l H_{t-1} + k_t v_t^T,   o_t = scale * H_t^T q_t
//
// One CTA of 128 threads per (value head, sequence); thread j keeps column j of H in
// registers and walks the tokens, q and k of 16 tokens at a time staged in shared memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include "decay_common.cuh"
#include "gdr_common.cuh"
#include "gdr_host.h"

namespace gdr {
namespace {

constexpr int D = kHeadDim;
constexpr int kBlock = 16;   // tokens staged at a time

struct DecayPrefillParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *log_decay;
  float scale;
  int hv, group;
  const int32_t *cu;
  DecayStates st;
  uint16_t *o;
};

__global__ void __launch_bounds__(D) decay_prefill_kernel(DecayPrefillParams p) {
  const int h = blockIdx.x, n = blockIdx.y, j = threadIdx.x;
  __shared__ float s_q[kBlock][D], s_k[kBlock][D];
  grid_dep_wait();
  grid_dep_launch();
  const float *in;
  float *out;
  p.st.resolve(n, h, p.hv, &in, &out);
  float H[D];
#pragma unroll
  for (int i = 0; i < D; ++i) H[i] = in ? in[i * D + j] : 0.0f;
  const DecayStep st = decay_step(p.log_decay[h], 1);
  const int kh = h / p.group;
  const int64_t t0 = p.cu[n], t1 = p.cu[n + 1];
  for (int64_t t = t0; t < t1; t += kBlock) {
    const int m = t1 - t < kBlock ? static_cast<int>(t1 - t) : kBlock;
    __syncthreads();
    for (int r = 0; r < m; ++r) {
      s_q[r][j] = bf_bits2f(p.q[(t + r) * p.q_stride + kh * D + j]);
      s_k[r][j] = bf_bits2f(p.k[(t + r) * p.k_stride + kh * D + j]);
    }
    __syncthreads();
    for (int r = 0; r < m; ++r) {
      const float v = bf_bits2f(p.v[(t + r) * p.v_stride + h * D + j]);
      float acc = 0.0f;
#pragma unroll
      for (int i = 0; i < D; ++i) {
        H[i] = st.apply(H[i], s_k[r][i] * v);
        acc += s_q[r][i] * H[i];
      }
      p.o[((t + r) * p.hv + h) * D + j] = f2bf_bits(p.scale * acc);
    }
  }
  if (out) {
#pragma unroll
    for (int i = 0; i < D; ++i) out[i * D + j] = H[i];
  }
}

}  // namespace

size_t decay_prefill_workspace_bytes(const int32_t *, int, int) { return 0; }

int launch_decay_prefill(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                         int64_t v_stride, const float *log_decay, float scale, int hk, int hv,
                         const int32_t *cu_dev, const int32_t *, int n_seqs, const DecayStates &states, void *o,
                         void *, cudaStream_t s) {
  DecayPrefillParams p;
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.log_decay = log_decay;
  p.scale = scale;
  p.hv = hv;
  p.group = hv / hk;
  p.cu = cu_dev;
  p.st = states;
  p.o = static_cast<uint16_t *>(o);
  return launch_status(launch_pdl(decay_prefill_kernel, dim3(hv, n_seqs), dim3(D), 0, s, 1, p),
                       "decay prefill: kernel launch");
}

}  // namespace gdr

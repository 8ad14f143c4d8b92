// The whole MoE layer for a few tokens (T <= 16) in one launch.
//
// A decode step reads the weights of the experts it routes to and little
// else, so the layer is a stream of weights with a few rows of activations:
// memory bound, and with eight launches between which nothing streams, latency
// bound too. Here one cooperative kernel, one block per SM, does all of it:
//
//   1. router: every block takes a few (token, expert) logits, fp32 dot
//      products, and brings the tokens' rows into shared memory; grid barrier;
//      every block takes the top-k of all tokens itself (the same arithmetic
//      everywhere) and lists the experts with rows.
//   2. mlp1: the active experts' hidden units, 8 at a time (a granule: 8 gate
//      rows and the 8 up rows of W1), are split evenly over the blocks; h
//      (bf16, rows by expert) goes to the workspace; grid barrier.
//   3. mlp2: granules of 16 rows of W2, split the same way; the fp32 expert
//      outputs go to the workspace; grid barrier;
//   4. combine: the k terms of every output element in slot order.
//
// A granule is 16 weight rows by the whole reduction. The block's 16 warps
// split the reduction, so that every SM has work for as little as one token
// and each warp meets the same slice of the activations in every granule.
// The rings run on across granules, experts and from mlp1 into mlp2, whose
// first weights arrive while the grid barrier is waited for. The multiplication
// is mma.sync m16n8k16: the 16 weight rows are M, up to 8 tokens are N (two N
// halves for more than 8). That is the shape this work has -- a 128-row tensor
// tile would leave the SMs unevenly loaded -- and the tensor rate is far from
// being a limit. The k index of an MMA is permuted (lane q of a row's four holds
// 8 consecutive elements of a 32-element unit), the same for weights and
// activations, so that the activations are read with wide shared-memory loads. The
// warps' partial sums meet in shared memory behind mbarriers (full / empty per
// buffer): some of the warps add them in warp order and finish the granule a turn
// later.
//
// bf16: each warp streams its own slices through its own cp.async ring, with no
// synchronisation between the warps to load.
//
// MXFP4: the granules are a quarter of the size and the work on a byte four
// times as much, so instructions and hand-overs count: other warps bring pairs
// of granules in by bulk copies (the 16 spend nothing on loads), and the warps
// work on four granules at a time (a turn), four on each, which leaves fewer
// partial sums to add (two granules a turn: 81 -> 92 us for 7 tokens). A unit of 32 codes is one scale block. The codes
// become f16 (exact), the activations f16 with one power of two per row such that
// the largest magnitude is in [2^8, 2^9) (exact down to 2^-25 of it, absolute
// error below 2^-33 of it), and each unit's fp32 sum is added with its weight
// scale. An expert with one or two tokens, the usual case of a decode step, would
// leave most columns of an MMA empty: the columns then hold the activations of 4
// units (of 2 for three or four tokens), loaded once for all of them, and each
// unit's MMA is right in its own columns (that and ldmatrix for the codes: 8
// tokens, D = 4096, I = 1536, 64 experts 68 -> 58 us).
//
// All sums are fp32. The order is fixed by the sizes, so results are bitwise
// reproducible.
//
// Measured, D = I = 2880, top-4 (the weights' bytes at the measured copy rate in
// brackets; a kernel that only reads needs 36 us for one token's 199 MB of bf16
// weights and about 15 for its 53 MB of MXFP4): 32 experts, bf16, 1 token 48 us
// (30), 16 tokens 239 to 257 (212 to 235); MXFP4, 1 token 27 us (8); 128 experts,
// MXFP4, 7 tokens 75 to 83 us (50 to 56). What is left: about 5 us in front of one
// token's weights (9 for 7 tokens and 128 experts: router, barrier, lists), 2 us at
// each later barrier and 2 to 4 of SMs that end unequally; MXFP4 turns take 2.2 us,
// what the memory needs, but mlp2's first, which also brings the rows of h, ends 6.5
// us after the barrier. The loop over the two weights is unrolled, 81 -> 78 us,
// although every SM then fetches another code for mlp2. Codes copied row by row are
// further from the memory's rate: 8 tokens, D = I = 4096, 7 of 8 experts 65 us (28),
// D = 7168, I = 2048, 21 of 32 experts 146 us (76). Measured and not kept: 24 warps
// for MXFP4 (72 registers: no faster), a granule a stage (94 -> 108 us: twice the
// hand-overs), codes without bank conflicts by exchanging units in registers (94 ->
// 102: the shared memory is not what bounds), two granules per warp sharing the
// activations' loads (mlp1 41 -> 49 us), row-by-row copies of codes that lie well
// (60 ns each: 49 -> 60), a router worked out by every block in place of the first
// barrier (4.1 -> 10.9 us: every SM reads the same weights from cold).
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;             // that compute
constexpr int kLoaders = 4;            // that load, in an MXFP4 block
constexpr int kThreads = kWarps * 32;
// Registers per thread of an MXFP4 block's loading and computing warps, out of
// the 96 that 640 threads are launched with.
constexpr int kRegsLaunch = 65536 / (kThreads + 32 * kLoaders) / 8 * 8, kRegsLoad = 32;
constexpr int kRegsCompute = (kRegsLaunch * (kThreads + 32 * kLoaders) - kRegsLoad * 32 * kLoaders) / kThreads / 8 * 8;
static_assert(kLoaders == 4 && kRegsCompute > kRegsLaunch, "");
constexpr int kMaxT = 16;
constexpr int kMaxK = 8;
constexpr int kMaxActive = kMaxT * kMaxK;
constexpr int kMaxSmem = 232448;      // 227 KB per block
constexpr int kStaticSmem = 4096;     // of it for FewShared
constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 4;
constexpr int64_t kMaxRowBytes = 65536 * 2;  // T * max(D, I) bf16 of resident activations
constexpr uint64_t kBarrierNs = 1000000000ull;

// Grid-barrier counters in the workspace header (the status word is at byte
// 0), as 32-bit words: blocks that reached each of the barriers, and blocks that
// are done.
constexpr int kBar1 = 16, kBar2 = 24, kBar3 = 32, kExit = 40;

// bf16 rings: a stage is 2 units of 32 of 16 rows, 128 bytes of a row, with
// the 16-byte pieces swizzled by row parity.
constexpr int kBfUnits = 2, kBfPitch = 128, kBfSlot = 16 * kBfPitch;
// MXFP4 ring: a stage is two neighbouring granules, or their part over a chunk
// of the reduction where they are too large for it.

struct FewParams {
  int T, D, E, k, I;
  const uint16_t *x, *Wr, *br, *b1, *b2;
  const uint8_t *w1, *w2, *s1, *s2;
  float* logits;     // (T, E)
  uint16_t* h;       // (T*k, I) bf16, rows by expert
  float* o;          // (T*k, D) fp32, by assignment, gate weight applied
  uint16_t* y;
  unsigned* header;  // workspace header
  int stages;        // of a warp's bf16 ring, or of the block's MXFP4 ring
  int slab_bytes;    // MXFP4: a stage
  int nchunks1, nchunks2;  // MXFP4: parts of the reduction of W1's and W2's stages
  int red_bufs;      // buffers for the warps' partial sums: 4, or 2 or 1 where shared memory is short
  int row_pitch;     // bytes between resident activation rows
  Act act;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// All but the newest n groups have landed.
__device__ __forceinline__ void cp_wait_upto(int n) {
  switch (n) {
    case 1: cp_wait<1>(); break;
    case 2: cp_wait<2>(); break;
    case 3: cp_wait<3>(); break;
    case 4: cp_wait<4>(); break;
    case 5: cp_wait<5>(); break;
    case 6: cp_wait<6>(); break;
    case 7: cp_wait<7>(); break;
    default: cp_wait<0>(); break;
  }
}

// Shared memory is read through ordinary pointers and the MMAs are not volatile,
// so that the loads of later units can be scheduled above the MMAs of earlier ones.
template <class T>
__device__ __forceinline__ T lds(const uint8_t* at) {
  return *reinterpret_cast<const T*>(at);
}

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with f16 operands, D apart from C.
__device__ __forceinline__ void mma_f16_16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 E2M1 codes (low nibble first) -> 4 pairs of f16.
__device__ __forceinline__ void e2m1_to_f16(uint32_t codes, uint32_t (&p)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
      : "r"(codes));
}

// E8M0: 2^(s - 127); the smallest, 2^-127, counts as zero.
__device__ __forceinline__ float e8m0(uint32_t s) { return __uint_as_float(s << 23); }

// The 16 computing warps meet (an MXFP4 block has more, which load).
__device__ __forceinline__ void warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

__device__ __forceinline__ void loaders_sync() { asm volatile("bar.sync 2, %0;" ::"n"(32 * kLoaders) : "memory"); }

// All blocks of the grid meet (the launch is cooperative, so all are
// resident): each arrives, and waits for the others at most kBarrierNs, then
// records the timeout and goes on -- every index computed later is in range
// whatever the data hold.
__device__ __forceinline__ void grid_arrive(unsigned* header, int which) {
  warps_sync();
  if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(header + which) : "memory");
}
__device__ __forceinline__ void grid_wait(unsigned* header, int which) {
  if (threadIdx.x == 0) {
    unsigned seen;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(header + which) : "memory");
      if (seen >= gridDim.x) break;
      if ((i & 63u) == 0) {
        const uint64_t now = sm100::globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kBarrierNs) {
          record_status(reinterpret_cast<int*>(header), MOE_ERR_TIMEOUT);
          break;
        }
      }
    }
  }
  warps_sync();
}
__device__ __forceinline__ void grid_barrier(unsigned* header, int which) {
  grid_arrive(header, which);
  grid_wait(header, which);
}

// The last block to leave sets the counters back to zero for the next call
// (every block has then passed the barriers, or given up on them).
__device__ __forceinline__ void grid_exit(unsigned* header) {
  if (threadIdx.x == 0 && atomicAdd(header + kExit, 1u) == gridDim.x - 1) {
    header[kBar1] = 0;
    header[kBar2] = 0;
    header[kBar3] = 0;
    header[kExit] = 0;
  }
}

// Order-preserving integer of a logit; NaN sorts below every number, -0 as +0.
__device__ __forceinline__ uint32_t sort_key(float v) {
  if (!(v == v)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  if (key == 0u) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

struct FewShared {
  uint64_t full[kMaxBufs], empty[kMaxBufs];        // of the partial-sum buffers
  uint64_t w_full[kMaxStages], w_empty[kMaxStages];  // of the MXFP4 ring
  int gave_up;                   // a wait of this block ran out of time
  int n_active;
  uint32_t tokens[256];          // per expert: its tokens, a bit each
  uint8_t place[256];            // per expert: its place among the active ones
  uint8_t expert[kMaxActive];    // active experts, ascending
  uint8_t start[kMaxActive + 1]; // first row of each active expert
  uint8_t slot[kMaxActive];      // per row: its assignment t * k + j
  uint8_t top[kMaxT][kMaxK];     // expert of each assignment
  uint8_t token[kMaxActive];     // per row
  float gate[kMaxActive];        // per assignment
  float dot[kWarps];
  uint32_t row_max[kMaxT];       // |largest| of each resident row (bf16 bits)
  float row_scale[kMaxT];        // what a resident row's sums are multiplied with
};

// Wait for a phase of an mbarrier, kBarrierNs at most, or until the block has
// given up elsewhere. The clock is looked at only now and then: reading it takes
// as long as these waits mostly last.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const volatile int* gave_up) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !sm100::mbar_try_wait(bar, parity); ++i) {
    if ((i & 255u) == 0) {
      if (gave_up && *gave_up) return false;
      const uint64_t now = sm100::globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kBarrierNs) return false;
    }
  }
  return true;
}

// Wait inside the block for warps that are on their way.
__device__ __forceinline__ void wait_local(uint32_t bar, uint32_t parity, FewShared& sh, unsigned* header) {
  if (!wait_bounded(bar, parity, &sh.gave_up)) {
    record_status(reinterpret_cast<int*>(header), MOE_ERR_TIMEOUT);
    *static_cast<volatile int*>(&sh.gave_up) = 1;
  }
}

static_assert(sizeof(FewShared) <= kStaticSmem, "");

// MXFP4: units per stage of a granule, even (K is a multiple of 64).
__host__ __device__ constexpr int mx_chunk(int units, int nchunks) {
  return ((units + nchunks - 1) / nchunks + 1) / 2 * 2;
}
// Bytes between a stage's rows of codes. Rows 32 or 96 bytes off a multiple of
// 128 collide two ways at most and are copied as they lie, a granule's 8 or 16
// at a time (a bulk copy costs its issuer some 60 ns whatever its size); others
// are copied row by row to an odd multiple of 16 (no collision).
__host__ __device__ constexpr bool mx_as_stored(int units, int nchunks) { return nchunks == 1 && units % 4 == 2; }
__host__ __device__ constexpr int mx_pitch(int units, int nchunks, int chunk) {
  return mx_as_stored(units, nchunks) ? units * 16 : (chunk | 1) * 16;
}
// A stage: 32 rows of codes, then all of the 32 rows' scales (with every chunk).
__host__ __device__ constexpr int mx_stage_bytes(int units, int nchunks) {
  return (32 * (mx_pitch(units, nchunks, mx_chunk(units, nchunks)) + units) + 127) / 128 * 128;
}

// log2 of the warps that split a granule's reduction, and the granules that the
// block works on at a time (a turn).
template <int kFmt>
constexpr int kSplitLog2 = kFmt == MOE_W_BF16 ? 4 : 2;
template <int kFmt>
constexpr int kTurn = kWarps >> kSplitLog2<kFmt>;

// One weight's granules as this block and warp see them.
struct Stream {
  int64_t row_bytes;     // of the weight
  int srow_bytes;        // of its scales
  int rows;              // weight rows per expert
  int up;                // row of the 9th weight row relative to the 1st (I: the up half; 8)
  int step;              // weight rows a granule advances by (8 or 16)
  int per_expert;        // granules per expert
  int side, part;        // this warp's granule of a turn, its part of the granule's reduction
  int u0, u1;            // this warp's units of 32 of the reduction
  int units;             // units of the reduction
  int nchunks;           // stages per granule
  int chunk;             // MXFP4: units per stage
  int g0, g1;            // this block's granules, over the active experts
};

template <int kFmt>
__device__ __forceinline__ Stream make_stream(const FewParams& p, int which, int n_active, int warp) {
  Stream s;
  const int K = which == 1 ? p.D : p.I;
  s.units = K / 32;
  s.row_bytes = kFmt == MOE_W_BF16 ? 2 * K : K / 2;
  s.srow_bytes = K / 32;
  s.rows = which == 1 ? 2 * p.I : p.D;
  s.up = which == 1 ? p.I : 8;
  s.step = which == 1 ? 8 : 16;
  s.per_expert = which == 1 ? p.I / 8 : p.D / 16;
  const uint32_t n = n_active * s.per_expert;  // at most 128 * 2048
  s.g0 = static_cast<int>(n * blockIdx.x / gridDim.x);
  s.g1 = static_cast<int>(n * (blockIdx.x + 1) / gridDim.x);
  s.side = warp >> kSplitLog2<kFmt>;
  s.part = warp & ((1 << kSplitLog2<kFmt>) - 1);
  // bf16: this warp's units, two a stage
  const int per = (s.units + (1 << kSplitLog2<kFmt>) - 1) >> kSplitLog2<kFmt>;
  s.u0 = min(s.units, s.part * per);
  s.u1 = min(s.units, s.u0 + per);
  s.nchunks = kFmt == MOE_W_BF16 ? (per + kBfUnits - 1) / kBfUnits : which == 1 ? p.nchunks1 : p.nchunks2;
  s.chunk = mx_chunk(s.units, s.nchunks);
  return s;
}

// The loading end of a warp's bf16 ring: where its next stage comes from, and
// which 16-byte pieces each lane copies.
struct Loader {
  uint32_t off[4];              // from the granule's first row, this warp's first unit
  const uint8_t* w;             // the current granule's first row
  int ai, local, end, chunk;    // active expert (-1: no more), granule, end of the expert's granules, stage

  // To the first granule `begin` of active expert ai.
  __device__ __forceinline__ void seek(const FewParams& p, const FewShared& sh, const Stream& st, int which,
                                       int begin) {
    if (ai * st.per_expert >= st.g1) {
      ai = -1;
      return;
    }
    end = min(st.per_expert, st.g1 - ai * st.per_expert);
    local = begin;
    w = (which == 1 ? p.w1 : p.w2) +
        (static_cast<int64_t>(sh.expert[ai]) * st.rows + static_cast<int64_t>(local) * st.step) * st.row_bytes;
  }

  __device__ __forceinline__ void start(const FewParams& p, const FewShared& sh, const Stream& st, int which,
                                        int lane) {
    chunk = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = lane + 32 * i, r = idx / 8, c = idx % 8;
      off[i] = static_cast<uint32_t>((r < 8 ? r : st.up + r - 8) * st.row_bytes + st.u0 * 64 + c * 16);
    }
    ai = -1;
    if (st.g0 < st.g1) {
      ai = st.g0 / st.per_expert;
      seek(p, sh, st, which, st.g0 % st.per_expert);
    }
  }

  // Copy this warp's part of the next stage into its ring slot.
  __device__ __forceinline__ void load(const FewParams& p, const FewShared& sh, const Stream& st, int which,
                                       uint32_t slot, int lane) {
    const int u = chunk * kBfUnits;  // from the warp's first unit
    const int valid = min(kBfUnits, st.u1 - st.u0 - u) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = lane + 32 * i, r = idx / 8, c = idx % 8;
      if (c < valid) cp_async16(slot + r * kBfPitch + (c ^ ((r & 1) << 2)) * 16, w + off[i] + u * 64);
    }
    if (++chunk == st.nchunks) {
      chunk = 0;
      if (++local < end) {
        w += st.step * st.row_bytes;
      } else {
        ++ai;
        seek(p, sh, st, which, 0);
      }
    }
  }
};

// The loading warps of an MXFP4 block: mlp1's granules then mlp2's, turn by
// turn, two granules a stage. Of W1 rows 0..15 of a stage are gate rows and
// 16..31 the up rows. The first warp does it alone where the codes are copied as
// they lie; row by row each of the four copies its quarter of the rows (four
// issuers of bulk copies reach twice the rate of one).
__device__ __forceinline__ void mx_produce(const FewParams& p, FewShared& sh, const Stream& st1, const Stream& st2,
                                           uint32_t ring, int loader, int lane) {
  using namespace sm100;
  const uint32_t full = smem_u32(sh.w_full), empty = smem_u32(sh.w_empty);
  int slot = 0, issued = 0;
  uint32_t phase = 0;
  bool failed = false;
  for (int which = 1; which <= 2; ++which) {
    // (the other loaders have not followed the ring's phases through a weight
    // that the first copies alone: they go on from where it stands)
    if (which == 2) loaders_sync();
    const Stream& st = which == 1 ? st1 : st2;
    const int pitch = mx_pitch(st.units, st.nchunks, st.chunk);
    const bool as_stored = mx_as_stored(st.units, st.nchunks), idle = as_stored && loader != 0;
    int ai = st.g0 / st.per_expert, local = st.g0 % st.per_expert;
    for (int g = st.g0; g < st.g1 && !failed;) {
      const int left = min(st.per_expert - local, st.g1 - g);  // of this expert
      const int count = min(2, left);
      // runs of neighbouring rows: W1's gate and up rows, W2's rows
      const int runs = which == 1 ? 2 : 1, run = count * (which == 1 ? 8 : 16);
      const int64_t row0 = static_cast<int64_t>(sh.expert[ai]) * st.rows + static_cast<int64_t>(local) * st.step;
      const uint8_t* w = (which == 1 ? p.w1 : p.w2) + row0 * st.row_bytes;
      const uint8_t* s = (which == 1 ? p.s1 : p.s2) + row0 * st.srow_bytes;
      for (int c = 0; c < st.nchunks; ++c) {
        if (!idle && !wait_bounded(empty + 8 * slot, phase ^ 1u, &sh.gave_up)) {
          failed = true;
          break;
        }
        const int n = min(st.chunk, st.units - c * st.chunk);
        const uint32_t bar = full + 8 * slot, to = ring + slot * p.slab_bytes;
        if (loader == 0 && lane == 0) mbar_arrive_expect_tx(bar, 16 * count * (n * 16 + st.srow_bytes));
        __syncwarp();
        if (loader == 0 && lane < runs)
          bulk_load(to + 32 * pitch + lane * 16 * st.srow_bytes, s + static_cast<int64_t>(lane) * st.up * st.srow_bytes,
                    run * st.srow_bytes, bar);
        if (as_stored) {
          if (loader == 0 && lane < runs)
            bulk_load(to + lane * 16 * pitch, w + lane * st.up * st.row_bytes, run * pitch, bar);
        } else {
          const int i = lane * kLoaders + loader, r = i % run;  // the lane's row, of the first 8 lanes
          if (i < runs * run)
            bulk_load(to + (i / run * 16 + r) * pitch, w + (r + i / run * st.up) * st.row_bytes + c * st.chunk * 16,
                      n * 16, bar);
        }
        ++issued;
        if (++slot == p.stages) {
          slot = 0;
          phase ^= 1u;
        }
      }
      g += count;
      local += count;
      if (local == st.per_expert) {
        local = 0;
        ++ai;
      }
    }
  }
  if (failed) {
    if (lane == 0) record_status(reinterpret_cast<int*>(p.header), MOE_ERR_TIMEOUT);
    *static_cast<volatile int*>(&sh.gave_up) = 1;
    // the copies still in flight land before the block can exit
    for (int i = min(issued, p.stages); i > 0; --i) {
      if (--slot < 0) {
        slot = p.stages - 1;
        phase ^= 1u;
      }
      wait_bounded(full + 8 * slot, phase, nullptr);
    }
  }
}

// acc (the first kG of kN groups of 8 tokens) += 16 weight rows x n <= 2 units of a bf16 stage.
// Two units of a row are 8 pieces of 16 bytes: piece 4 j + q, the halves
// exchanged in odd rows (conflict-free). `b`: the lane's place in its rows of
// the activations.
template <int kG, int kN>
__device__ __forceinline__ void mul_bf16(const uint8_t* slot, int r, int q, int n, const uint8_t* const (&b)[kN],
                                         float (&acc)[kN][4]) {
#pragma unroll
  for (int j = 0; j < kBfUnits; ++j) {
    if (j < n) {
      const uint8_t* at = slot + r * kBfPitch + (((4 * j + q) ^ ((r & 1) << 2)) * 16);
      const uint4 a = lds<uint4>(at), a8 = lds<uint4>(at + 8 * kBfPitch);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const uint4 v = lds<uint4>(b[g] + j * 64);
        mma_bf16_16816(acc[g], a.x, a8.x, a.y, a8.y, v.x, v.y);
        mma_bf16_16816(acc[g], a.z, a8.z, a.w, a8.w, v.z, v.w);
      }
    }
  }
}

// Four 8 x 16-byte matrices of shared memory, whose rows the lanes 8 m + i point
// at: register m of lane 4 r + q holds bytes 4 q.. of row r of matrix m.
__device__ __forceinline__ void ldmatrix_x4(uint32_t at, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(at));
}

// The same for kUnits (even) units of MXFP4 codes, with the columns of an MMA's
// activations shared by kPack units, 8 / kPack tokens each: one load of the
// activations serves them all, and of each unit's sums a quarter of the lanes, or
// a half, are its own -- those lanes bring its scale and add them (the others hold
// products of one unit's codes with another's activations). at: the row of codes
// that this lane points at for two units of the granule's first and last 8 rows;
// s_lo, s_hi: the lane's place in its two rows' scales (of its own unit of the
// kPack); own: which of them that is. All of them and b move on.
template <int kG, int kUnits, int kPack, int kN>
__device__ __forceinline__ void mul_mx(uint32_t& at, const uint8_t*& s_lo, const uint8_t*& s_hi,
                                       const uint8_t* (&b)[kN], int own, const float (&zero)[4], float (&acc)[kN][4]) {
  constexpr int kStep = kPack > 2 && kUnits > 2 ? 4 : 2;  // units that are begun together
#pragma unroll
  for (int j = 0; j < kUnits; j += kStep) {
    uint4 x[kG];
    uint32_t w_lo, w_hi;
    if (kPack == 1) {
      w_lo = lds<uint16_t>(s_lo + j);
      w_hi = lds<uint16_t>(s_hi + j);
    } else {
      w_lo = lds<uint8_t>(s_lo + j);
      w_hi = lds<uint8_t>(s_hi + j);
#pragma unroll
      for (int g = 0; g < kG; ++g) x[g] = lds<uint4>(b[g] + j * 64);
    }
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      if (i % 2 == 0) ldmatrix_x4(at + (j + i) * 16, v);
      uint32_t a[4], a8[4];
      e2m1_to_f16(v[i % 2], a);
      e2m1_to_f16(v[2 + i % 2], a8);
      const float f_lo = e8m0(kPack > 1 ? w_lo : i == 0 ? w_lo & 0xffu : w_lo >> 8);
      const float f_hi = e8m0(kPack > 1 ? w_hi : i == 0 ? w_hi & 0xffu : w_hi >> 8);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        if (kPack == 1) x[g] = lds<uint4>(b[g] + (j + i) * 64);
        float c[4];
        mma_f16_16816_from(c, a[0], a8[0], a[1], a8[1], x[g].x, x[g].y, zero);
        mma_f16_16816(c, a[2], a8[2], a[3], a8[3], x[g].z, x[g].w);
        if (kPack == 1 || own == i) {
          acc[g][0] = fmaf(f_lo, c[0], acc[g][0]);
          acc[g][1] = fmaf(f_lo, c[1], acc[g][1]);
          acc[g][2] = fmaf(f_hi, c[2], acc[g][2]);
          acc[g][3] = fmaf(f_hi, c[3], acc[g][3]);
        }
      }
    }
  }
  at += kUnits * 16;
  s_lo += kUnits;
  s_hi += kUnits;
#pragma unroll
  for (int g = 0; g < kG; ++g) b[g] += kUnits * 64;
}
// The same for `left` units, an even number, of one group of tokens.
template <int kPack, int kN>
__device__ __forceinline__ void mul_mx_row(int left, uint32_t at, const uint8_t* s_lo, const uint8_t* s_hi,
                                           const uint8_t* (&b)[kN], int own, const float (&zero)[4],
                                           float (&acc)[kN][4]) {
  for (; left >= 8; left -= 8) mul_mx<1, 8, kPack>(at, s_lo, s_hi, b, own, zero, acc);
  if (left & 4) mul_mx<1, 4, kPack>(at, s_lo, s_hi, b, own, zero, acc);
  if (left & 2) mul_mx<1, 2, kPack>(at, s_lo, s_hi, b, own, zero, acc);
}

// Bring `rows` rows of K bf16 into shared memory; MXFP4 rows become f16
// scaled by a power of two. row_max is zero on entry, and the warps
// synchronise before they read the rows. kHere: the rows are in shared memory
// already, where each thread has copied the pieces that it handles here.
template <int kFmt, bool kHere>
__device__ __forceinline__ void load_rows(const FewParams& p, FewShared& sh, const uint16_t* from, int rows, int K,
                                          uint8_t* act) {
  const int per = K / 8;  // 16-byte chunks per row
  constexpr int kAtOnce = 4;  // rows in flight
  for (int n0 = 0; n0 < rows; n0 += kAtOnce) {
    for (int base = threadIdx.x & ~31; base < per; base += kThreads) {  // (uniform in a warp)
      const int c = base + (threadIdx.x & 31);
      uint4 v[kAtOnce];
#pragma unroll
      for (int z = 0; z < kAtOnce; ++z) {
        v[z] = make_uint4(0, 0, 0, 0);
        if (n0 + z < rows && c < per)
          v[z] = kHere ? lds<uint4>(act + (n0 + z) * p.row_pitch + c * 16)
                       : __ldcg(reinterpret_cast<const uint4*>(from) + static_cast<int64_t>(n0 + z) * per + c);
      }
#pragma unroll
      for (int z = 0; z < kAtOnce; ++z) {
        if (n0 + z >= rows) break;
        if (!kHere && c < per) *reinterpret_cast<uint4*>(act + (n0 + z) * p.row_pitch + c * 16) = v[z];
        if (kFmt == MOE_W_MXFP4) {
          const uint32_t w[4] = {v[z].x, v[z].y, v[z].z, v[z].w};
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
          m = __reduce_max_sync(0xffffffffu, m);
          if ((threadIdx.x & 31) == 0) atomicMax(&sh.row_max[n0 + z], m);
        }
      }
    }
  }
  if (kFmt == MOE_W_MXFP4) {
    warps_sync();
    for (int n0 = 0; n0 < rows; n0 += kAtOnce) {
      float mul[kAtOnce];
#pragma unroll
      for (int z = 0; z < kAtOnce; ++z) {
        // 2^shift brings the row's largest magnitude into [2^8, 2^9); with an
        // infinity or NaN the largest there can be beside it, so that finite
        // values do not become infinite in f16; a row of zeros stays as it is
        const int n = min(n0 + z, rows - 1);
        const uint32_t largest = sh.row_max[n];
        const int ex = min(static_cast<int>(largest >> 7), 254);  // biased exponent
        const int shift = largest == 0 ? 0 : min(127, 8 + 127 - max(ex, 1));
        mul[z] = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
        if (threadIdx.x == 0)
          sh.row_scale[n] = __uint_as_float(shift == 127 ? 0x00400000u : static_cast<uint32_t>(127 - shift) << 23);
      }
      for (int c = threadIdx.x; c < per; c += kThreads) {
        uint8_t* at = act + n0 * p.row_pitch + c * 16;
        uint4 v[kAtOnce];
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z)
          if (n0 + z < rows) v[z] = lds<uint4>(at + z * p.row_pitch);
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z) {
          if (n0 + z >= rows) break;
          uint32_t w[4] = {v[z].x, v[z].y, v[z].z, v[z].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 h2 = __floats2half2_rn(__uint_as_float(w[i] << 16) * mul[z],
                                                 __uint_as_float(w[i] & 0xffff0000u) * mul[z]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          *reinterpret_cast<uint4*>(at + z * p.row_pitch) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
}

template <int kFmt, int kN>
__global__ void __launch_bounds__(kThreads + (kFmt == MOE_W_MXFP4 ? 32 * kLoaders : 0), 1)
    few_kernel(const FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  // resident rows | partial sums | rings
  uint8_t* act = smem;
  float* red = reinterpret_cast<float*>(smem + p.T * p.row_pitch);
  constexpr int kRedFloats = kWarps * 128 * kN;
  constexpr int kSplit = kSplitLog2<kFmt>;
  uint8_t* ring = reinterpret_cast<uint8_t*>(red + p.red_bufs * kRedFloats);
  __shared__ FewShared sh;

  // (the shuffle tells the compiler that the warp index is uniform)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0), lane = threadIdx.x % 32;

  if (kFmt == MOE_W_MXFP4) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.stages; ++i) {
        sm100::mbar_init(sm100::smem_u32(&sh.w_full[i]), 1);
        sm100::mbar_init(sm100::smem_u32(&sh.w_empty[i]), kWarps);
      }
      sm100::fence_mbar_init();
    }
    if (warp >= kWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
      __syncthreads();  // the lists are complete
      mx_produce(p, sh, make_stream<kFmt>(p, 1, sh.n_active, 0), make_stream<kFmt>(p, 2, sh.n_active, 0),
                 sm100::smem_u32(ring), warp - kWarps, lane);
      return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
  }

  // ---- the tokens' rows are asked for (by the threads that look at them below);
  // router logits
  for (int n = 0; n < p.T; ++n)
    for (int c = threadIdx.x; c < p.D / 8; c += kThreads)
      cp_async16(sm100::smem_u32(act + n * p.row_pitch + c * 16), p.x + static_cast<int64_t>(n) * p.D + c * 8);
  cp_commit();
  if (threadIdx.x < 256) sh.tokens[threadIdx.x] = 0;
  if (threadIdx.x < kMaxT) sh.row_max[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    sh.gave_up = 0;
    for (int i = 0; i < kMaxBufs; ++i) {
      sm100::mbar_init(sm100::smem_u32(&sh.full[i]), kWarps);
      sm100::mbar_init(sm100::smem_u32(&sh.empty[i]), kWarps);
    }
    sm100::fence_mbar_init();
  }
  {
    // this block's logits, each by 16 / groups warps (one warp when there are
    // many), their parts added in warp order
    const uint32_t items = p.T * p.E;
    const int i0 = static_cast<int>(items * blockIdx.x / gridDim.x);
    const int n = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x) - i0;
    int groups = 1;
    while (groups < n && groups < kWarps) groups *= 2;
    const int parts = kWarps / groups, part = warp % parts;
    // the first weights are on their way while the tokens' rows arrive
    constexpr int kAhead = 6;
    const int step = parts * 32, c0 = part * 32 + lane;
    uint4 b[kAhead];
    auto ask = [&](int i, int c) {
      const uint4* from = reinterpret_cast<const uint4*>(p.Wr + static_cast<int64_t>((i0 + i) % p.E) * p.D);
#pragma unroll
      for (int z = 0; z < kAhead; ++z)
        if (c + z * step < p.D / 8) b[z] = __ldg(from + c + z * step);
    };
    int i = warp / parts;
    if (i < n) ask(i, c0);
    cp_wait<0>();
    warps_sync();
    for (bool asked = true; i < n; i += groups, asked = false) {
      const uint8_t* row = act + (i0 + i) / p.E * p.row_pitch;
      float sum = 0.0f;
      for (int c = c0; c < p.D / 8; c += kAhead * step) {
        if (!asked || c > c0) ask(i, c);
#pragma unroll
        for (int z = 0; z < kAhead; ++z) {
          if (c + z * step >= p.D / 8) break;
          const uint4 a = lds<uint4>(row + (c + z * step) * 16);
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b[z].x, b[z].y, b[z].z, b[z].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum = fmaf(__uint_as_float(aw[j] << 16), __uint_as_float(bw[j] << 16), sum);
            sum = fmaf(__uint_as_float(aw[j] & 0xffff0000u), __uint_as_float(bw[j] & 0xffff0000u), sum);
          }
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) {
        if (parts == 1)
          p.logits[i0 + i] = sum + bf16_bits_to_float(p.br[(i0 + i) % p.E]);
        else
          sh.dot[warp] = sum;
      }
    }
    warps_sync();
    if (parts > 1 && static_cast<int>(threadIdx.x) < n) {  // (then every logit had its own group)
      float sum = 0.0f;
      for (int i = 0; i < parts; ++i) sum += sh.dot[threadIdx.x * parts + i];
      const int at = i0 + threadIdx.x;
      p.logits[at] = sum + bf16_bits_to_float(p.br[at % p.E]);
    }
  }
  grid_arrive(p.header, kBar1);
  if constexpr (kFmt == MOE_W_MXFP4) load_rows<kFmt, true>(p, sh, p.x, p.T, p.D, act);  // while the others arrive
  grid_wait(p.header, kBar1);

  // ---- top-k of every token (warp t), then the active experts
  if (warp < p.T) {
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < p.E ? sort_key(__ldcg(p.logits + warp * p.E + e)) : 0u;
    }
    float first = 0.0f, total = 0.0f, mine = 0.0f;
    uint32_t taken = 0;  // bit i: this lane's expert lane + 32 i is chosen already
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (32 * i < p.E && !((taken >> i) & 1u)) best = max(best, key[i]);
      best = __reduce_max_sync(0xffffffffu, best);
      uint32_t at = 0xffffffffu;  // lowest expert that holds it and is not taken
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (32 * i < p.E && !((taken >> i) & 1u) && key[i] == best && lane + 32 * i < p.E) at = lane + 32 * i;
      at = __reduce_min_sync(0xffffffffu, at);
      if (static_cast<int>(at & 31u) == lane) taken |= 1u << (at >> 5);
      const float v = key_value(best);
      if (j == 0) first = v;
      const float ex = __expf(v - first);
      total += ex;
      if (lane == j) {
        mine = ex;
        sh.top[warp][j] = static_cast<uint8_t>(at);
        atomicOr(&sh.tokens[at], 1u << warp);
      }
    }
    if (lane < p.k) sh.gate[warp * p.k + lane] = __fdividef(mine, total);
  }
  warps_sync();
  if (warp == 0) {
    // experts 8 lane .. 8 lane + 7; active experts and rows before them
    uint32_t mask[8];
    int n = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mask[i] = sh.tokens[8 * lane + i];
      n += mask[i] != 0;
      rows += __popc(mask[i]);
    }
    int both = n << 16 | rows;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, both, off);
      if (lane >= off) both += v;
    }
    n = (both >> 16) - n;
    rows = (both & 0xffff) - rows;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (mask[i] == 0) continue;
      sh.place[8 * lane + i] = static_cast<uint8_t>(n);
      sh.expert[n] = static_cast<uint8_t>(8 * lane + i);
      sh.start[n++] = static_cast<uint8_t>(rows);
      rows += __popc(mask[i]);
    }
    if (lane == 31) {
      sh.n_active = n;
      sh.start[n] = static_cast<uint8_t>(rows);
    }
  }
  warps_sync();
  if (static_cast<int>(threadIdx.x) < p.T * p.k) {
    const int t = threadIdx.x / p.k, e = sh.top[t][threadIdx.x % p.k];
    const int row = sh.start[sh.place[e]] + __popc(sh.tokens[e] & ((1u << t) - 1u));
    sh.slot[row] = static_cast<uint8_t>(threadIdx.x);
    sh.token[row] = static_cast<uint8_t>(t);
  }
  const int n_active = sh.n_active;

  // ---- the weight stream: mlp1's stages, then mlp2's, through this warp's ring
  const Stream st1 = make_stream<kFmt>(p, 1, n_active, warp);
  const Stream st2 = make_stream<kFmt>(p, 2, n_active, warp);
  const uint8_t* ring_mine = ring + warp * p.stages * kBfSlot;  // bf16
  const uint32_t ring_at = sm100::smem_u32(ring_mine);
  Loader ld;
  if (kFmt == MOE_W_BF16) ld.start(p, sh, st1, 1, lane);
  int ld_which = 1, ld_slot = 0;
  auto issue = [&]() {
    if (ld_which == 1 && ld.ai < 0) {
      ld_which = 2;
      ld.start(p, sh, st2, 2, lane);
    }
    if (ld.ai >= 0) ld.load(p, sh, ld_which == 1 ? st1 : st2, ld_which, ring_at + ld_slot * kBfSlot, lane);
    cp_commit();
    if (++ld_slot == p.stages) ld_slot = 0;
  };
  if (kFmt == MOE_W_BF16)
    for (int i = 0; i < p.stages; ++i) issue();
  __syncthreads();  // the lists are complete

  // Four registers of zeros that the compiler takes for values: C of every
  // unit's first MMA, without writing zeros for each.
  float zero[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("mov.f32 %0, 0f00000000;" : "=f"(zero[i]));
  int slot = 0, it = 0;     // of the ring; turn
  uint32_t slab_phase = 0;  // MXFP4: of the ring
  const int buf_shift = p.red_bufs >> 1;  // log2 of 1, 2 or 4
  const uint32_t full_at = sm100::smem_u32(sh.full), empty_at = sm100::smem_u32(sh.empty);
  const int fr = lane / 4, fq = lane % 4;
#pragma unroll
  for (int which = 1; which <= 2; ++which) {
    const Stream& s = which == 1 ? st1 : st2;
    if (which == 2) grid_barrier(p.header, kBar2);  // h is complete
    const int pitch = mx_pitch(s.units, s.nchunks, s.chunk);
    for (int ai = s.g0 / s.per_expert; s.g0 < s.g1 && ai * s.per_expert < s.g1; ++ai) {
      const int begin = max(0, s.g0 - ai * s.per_expert), end = min(s.per_expert, s.g1 - ai * s.per_expert);
      const int e = sh.expert[ai], start = sh.start[ai], rows = sh.start[ai + 1] - start;
      if (which == 2) {
        warps_sync();  // the previous expert's rows are read no more
        if (threadIdx.x < kMaxT) sh.row_max[threadIdx.x] = 0;
        warps_sync();
        load_rows<kFmt, false>(p, sh, p.h + static_cast<int64_t>(start) * p.I, rows, p.I, act);
        warps_sync();
      }
      // MXFP4: up to 2 tokens share an MMA's columns with 4 units, up to 4 tokens
      // with 2 (wide: log2 of the lanes of a row's four that a token's unit has; own:
      // this lane's unit of the 4 or 2)
      const int wide = kFmt == MOE_W_BF16 || rows > 4 ? 2 : rows > 2 ? 1 : 0, own = fq >> wide;
      // a column without a token repeats the last row; its sums are not used
      const uint8_t* brow[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int n = min(8 * i + (fr & ((2 << wide) - 1)), rows - 1);
        brow[i] = act + (which == 1 ? sh.token[start + n] : n) * p.row_pitch + fq * 16 +
                  (kFmt == MOE_W_BF16 ? s.u0 * 64 : (fr >> (wide + 1)) * 64);
      }
      // A turn's granules are finished by some of the warps, each always with the
      // same task (every second, fourth, ... turn where there are fewer tasks than
      // warps), so what it needs is worked out once for the expert. A task is a sum a
      // lane: of a fragment's 128 elements 32, of those of the first of the 4 or 2
      // units, to which the others' are added. For more than 8 MXFP4 tokens it is a
      // whole fragment, four sums a lane, the units' added across the lanes, which
      // then share out the columns (9 tokens 121 -> 105 us, but 7 tokens 88 -> 92).
      constexpr bool kMx = kFmt == MOE_W_MXFP4, kWhole = kMx && kN == 2;
      constexpr int kCols = kWhole ? 2 : 1;  // tokens of a lane
      const int groups_log2 = kN == 1 || (kMx && rows <= 8) ? 0 : 1;
      const int quarters_log2 = kWhole ? 0 : wide;
      const int tasks_log2 = 4 - kSplit + groups_log2 + quarters_log2;
      const int turns_mask = (kWarps >> tasks_log2) - 1, my_turn = warp >> tasks_log2;
      const int id = warp & ((1 << tasks_log2) - 1);
      const int grp = (id >> quarters_log2) & ((1 << groups_log2) - 1), m = id >> (quarters_log2 + groups_log2);
      const bool mine = 8 * grp < rows;
      // the lane's first element of the fragment, and its weight row
      const int el = (id & ((1 << quarters_log2) - 1)) * 32 + lane, frag = el / 4;
      const int at = kWhole ? lane * 4 : ((frag >> wide) * 4 + (frag & ((1 << wide) - 1))) * 4 + el % 4;
      const int r = at / 16 + (at & 2 ? 8 : 0);
      const int pick = wide == 1 ? fq >> 1 : fq & 1;  // whole, up to 4 tokens: the lane's column of its two
      const float* const part = red + ((m << kSplit) * kN + grp) * 128 + at;
      const int bias_at = e * s.rows + (r < 8 ? r : s.up + r - 8);  // (at most 256 x 32768)
      const uint16_t* const bias_base = which == 1 ? p.b1 : p.b2;
      bool on[kCols];
      float scale[kCols], gate[kCols];
      int out[kCols];  // element of h or o, for granule 0 (rows of 16384 at most)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const int col = !kWhole     ? at / 4 % 4 * 2 + (at & 1)
                        : wide == 2 ? 2 * fq + c
                        : wide == 1 ? 2 * (fq & 1) + pick
                                    : pick;
        const int n = 8 * grp + col;
        // (an up half's lane of its own writes nothing: its gate's lane writes h)
        on[c] = mine && n < rows && (kWhole ? wide == 2 || (c == 0 && (wide == 1 || fq < 2)) : which == 2 || r < 8);
        const int row = start + (n < rows ? n : 0), a = sh.slot[row];
        scale[c] = kMx ? sh.row_scale[which == 1 ? sh.token[row] : row - start] : 1.0f;
        gate[c] = sh.gate[a];
        out[c] = (which == 1 ? row * p.I : a * p.D) + r;
      }
      uint16_t bias[2];
      // What the finish needs from memory, asked for a turn ahead.
      auto load_bias = [&](int first, int turn) {
        if ((turn & turns_mask) != my_turn || !mine || first + m >= end) return;
        bias[0] = bias_base[bias_at + (first + m) * s.step];
        if (kWhole) bias[1] = bias_base[bias_at + (first + m) * s.step + s.up];
      };
      auto finish = [&](int first, int turn) {
        const int buf = turn & (p.red_bufs - 1);
        const bool active = (turn & turns_mask) == my_turn;
        float sum[kWhole ? 4 : 1];
        if (active) {
          wait_local(full_at + 8 * buf, (turn >> buf_shift) & 1, sh, p.header);
#pragma unroll
          for (int c = 0; c < (kWhole ? 4 : 1); ++c) sum[c] = 0.0f;
          if (mine) {
            const float* from = part + buf * kRedFloats;
            if constexpr (kWhole) {
#pragma unroll 1
              for (int w = 0; w < 1 << kSplit; w += 4) {
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4*>(from + (w + i) * (kN * 128));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  sum[0] += v[i].x;
                  sum[1] += v[i].y;
                  sum[2] += v[i].z;
                  sum[3] += v[i].w;
                }
              }
            } else {
              for (int c = 0; c < 16; c += 4 << wide) {
#pragma unroll 4
                for (int w = 0; w < 1 << kSplit; ++w) sum[0] += from[w * (kN * 128) + c];
              }
            }
          }
          __syncwarp();
        }
        if (lane == 0) sm100::mbar_arrive(empty_at + 8 * buf);
        const int local = first + m;
        if (!active || !mine || local >= end) return;  // (uniform in a warp)
        if constexpr (kWhole) {
#pragma unroll
          for (int off = 2; off > 0; off /= 2)
            if (wide < off)
#pragma unroll
              for (int c = 0; c < 4; ++c) sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], off);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            if (c > 0 && wide < 2) break;
            const bool second = wide == 2 ? c > 0 : pick != 0;
            const float lo = fmaf(second ? sum[1] : sum[0], scale[c], bf16_bits_to_float(bias[0]));
            const float hi = fmaf(second ? sum[3] : sum[2], scale[c], bf16_bits_to_float(bias[1]));
            if (!on[c]) continue;
            if (which == 1) {
              p.h[out[c] + local * 8] = float_to_bf16_bits(glu_act(lo, hi, p.act));
            } else {
              p.o[out[c] + local * 16] = gate[c] * lo;
              p.o[out[c] + local * 16 + 8] = gate[c] * hi;
            }
          }
        } else {
          const float v = fmaf(sum[0], scale[0], bf16_bits_to_float(bias[0]));
          if (which == 1) {
            const float up = __shfl_xor_sync(0xffffffffu, v, 2);
            if (on[0]) p.h[out[0] + local * 8] = float_to_bf16_bits(glu_act(v, up, p.act));
          } else if (on[0]) {
            p.o[out[0] + local * 16] = gate[0] * v;
          }
        }
      };
      for (int base = begin; base < end; base += kTurn<kFmt>, ++it) {
        float acc[kN][4];
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
        if (kFmt == MOE_W_BF16) {
          for (int chunk = 0; chunk < s.nchunks; ++chunk) {
            cp_wait_upto(p.stages - 1);
            __syncwarp();
            const int u = chunk * kBfUnits;
            const uint8_t* b[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) b[i] = brow[i] + u * 64;
            if (kN == 1 || rows <= 8)
              mul_bf16<1>(ring_mine + slot * kBfSlot, fr, fq, s.u1 - s.u0 - u, b, acc);
            else
              mul_bf16<kN>(ring_mine + slot * kBfSlot, fr, fq, s.u1 - s.u0 - u, b, acc);
            __syncwarp();
            issue();
            if (++slot == p.stages) slot = 0;
          }
        } else {
          // Every warp waits for every stage of the turn, in order, and frees
          // it -- at once where its granule is not in it -- so that no slot's
          // phase passes a warp by.
          const int count = min(kTurn<kFmt>, end - base);
          for (int i = 0; i < (count + 1) / 2 * s.nchunks; ++i) {
            wait_local(sm100::smem_u32(&sh.w_full[slot]), slab_phase, sh, p.header);
            const int chunk = i - s.side / 2 * s.nchunks;
            if (chunk >= 0 && chunk < s.nchunks && s.side < count) {
              // this warp's units of the stage, an even number
              const int first = chunk * s.chunk, n = min(s.chunk, s.units - first);
              const int per = (n + (2 << kSplit) - 1) >> (kSplit + 1) << 1;
              const int u0 = min(n, s.part * per);
              int left = min(n, u0 + per) - u0;
              const uint8_t* slab = ring + slot * p.slab_bytes;
              const int lo = (which == 1 ? 8 : 16) * (s.side & 1), hi = lo + (which == 1 ? 16 : 8);  // its rows
              // codes: lanes 0..7 and 8..15 point at the first 8 rows, at one unit
              // and the next, 16..31 at the last 8
              uint32_t at = sm100::smem_u32(slab) + ((lane & 16 ? hi : lo) + (lane & 7)) * pitch +
                            (u0 + ((lane >> 3) & 1)) * 16;
              const uint8_t* s_lo = slab + 32 * pitch + (lo + fr) * s.srow_bytes + first + u0 + own;
              const uint8_t* s_hi = s_lo + (hi - lo) * s.srow_bytes;
              const uint8_t* b[kN];
#pragma unroll
              for (int j = 0; j < kN; ++j) b[j] = brow[j] + (first + u0) * 64;
              if (wide == 0) {
                mul_mx_row<4>(left, at, s_lo, s_hi, b, own, zero, acc);
              } else if (wide == 1) {
                mul_mx_row<2>(left, at, s_lo, s_hi, b, own, zero, acc);
              } else if (kN == 1 || rows <= 8) {
                mul_mx_row<1>(left, at, s_lo, s_hi, b, own, zero, acc);
              } else {
                for (; left >= 4; left -= 4) mul_mx<kN, 4, 1>(at, s_lo, s_hi, b, own, zero, acc);
                if (left) mul_mx<kN, 2, 1>(at, s_lo, s_hi, b, own, zero, acc);
              }
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sm100::smem_u32(&sh.w_empty[slot]));
            if (++slot == p.stages) {
              slot = 0;
              slab_phase ^= 1u;
            }
          }
        }
        // the warps' parts meet in buffer it mod red_bufs
        const int buf = it & (p.red_bufs - 1);
        float* part = red + buf * kRedFloats;
        if (it >= p.red_bufs) wait_local(empty_at + 8 * buf, ((it >> buf_shift) - 1) & 1, sh, p.header);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (i == 0 || rows > 8)
            *reinterpret_cast<float4*>(part + (warp * kN + i) * 128 + lane * 4) =
              make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(full_at + 8 * buf);
        // the previous granules are finished only now, when their parts are
        // all there; with one buffer these ones are, at once
        if (p.red_bufs == 1) {
          load_bias(base, it);
          finish(base, it);
        } else {
          if (base > begin) finish(base - kTurn<kFmt>, it - 1);
          load_bias(base, it);
        }
      }
      if (p.red_bufs > 1) finish(begin + (end - begin - 1) / kTurn<kFmt> * kTurn<kFmt>, it - 1);
    }
  }
  cp_wait<0>();

  // ---- combine: four columns of a token per thread, over the whole grid
  grid_barrier(p.header, kBar3);
  for (int i = blockIdx.x + threadIdx.x * gridDim.x; i < p.T * (p.D / 4); i += gridDim.x * kThreads) {
    const int t = i / (p.D / 4), c = i % (p.D / 4);
    const float4* from = reinterpret_cast<const float4*>(p.o + static_cast<int64_t>(t) * p.k * p.D) + c;
    float4 v[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (j < p.k) v[j] = __ldcg(from + static_cast<int64_t>(j) * (p.D / 4));
    float4 sum = v[0];
#pragma unroll
    for (int j = 1; j < kMaxK; ++j)
      if (j < p.k) sum = make_float4(sum.x + v[j].x, sum.y + v[j].y, sum.z + v[j].z, sum.w + v[j].w);
    *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(t) * p.D + 4 * c) =
        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
  }
  grid_exit(p.header);
}

template <int kFmt, int kN>
moe_status_t launch(FewParams p, cudaStream_t s) {
  constexpr bool mx = kFmt == MOE_W_MXFP4;
  const int red = kWarps * 128 * kN * 4;
  // (lanes whose unit of a shared MMA lies past the last one read up to 3 bytes past the last stage's scales)
  constexpr int past = 16;
  const int room = kMaxSmem - kStaticSmem - past - p.T * p.row_pitch;
  if (mx) {
    // as few parts of the reduction as let two stages fit where rows are copied
    // as they lie, else four (a turn takes two) unless the pieces get shorter
    // than 1 KB
    for (int which = 1; which <= 2; ++which) {
      const int units = (which == 1 ? p.D : p.I) / 32;
      auto wanted = [&](int n) { return !mx_as_stored(units, n) && (units + n - 1) / n > 64 ? 4 : 2; };
      int nchunks = 1;
      while (nchunks < units && wanted(nchunks) * mx_stage_bytes(units, nchunks) > room - red) ++nchunks;
      nchunks = (units + mx_chunk(units, nchunks) - 1) / mx_chunk(units, nchunks);
      (which == 1 ? p.nchunks1 : p.nchunks2) = nchunks;
      p.slab_bytes = std::max(p.slab_bytes, mx_stage_bytes(units, nchunks));
    }
  }
  const int stage = mx ? p.slab_bytes : kWarps * kBfSlot;
  // the most buffers for the partial sums that leave three stages, else two
  p.red_bufs = 0;
  for (int least = 3; least >= 2 && p.red_bufs == 0; --least)
    for (int bufs = kN == 1 ? 4 : 2; bufs >= 1 && p.red_bufs == 0; bufs /= 2)
      if (room - bufs * red >= least * stage) p.red_bufs = bufs;
  if (p.red_bufs == 0) return MOE_ERR_UNSUPPORTED;
  int stages = (room - p.red_bufs * red) / stage;
  if (stages > kMaxStages) stages = kMaxStages;
  p.stages = stages;
  const int smem = p.T * p.row_pitch + p.red_bufs * red + stages * stage + past;
  // (the same limit for every size: calls from several host threads do not meet another's)
  if (cudaFuncSetAttribute(few_kernel<kFmt, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMaxSmem - kStaticSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  void* args[] = {&p};
  if (cudaLaunchCooperativeKernel(reinterpret_cast<void*>(few_kernel<kFmt, kN>), dim3(num_sms()),
                                  dim3(kThreads + (mx ? 32 * kLoaders : 0)), args,
                                  smem, s) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace

int few_max_tokens(const moe_dims_t& d) {
  const int64_t wide = d.D > d.I ? d.D : d.I;
  const int64_t t = kMaxRowBytes / (2 * wide);
  return static_cast<int>(t < kMaxT ? t : kMaxT);
}

moe_status_t launch_few(const moe_dims_t& d, const uint16_t* x, const uint16_t* Wr, const uint16_t* br,
                        const moe_weight_t& W1, const uint16_t* b1, const moe_weight_t& W2, const uint16_t* b2,
                        uint16_t* y, float* logits, uint16_t* h, float* o, void* ws, cudaStream_t s) {
  FewParams p{};
  p.T = d.T;
  p.D = d.D;
  p.E = d.E;
  p.k = d.k;
  p.I = d.I;
  p.x = x;
  p.Wr = Wr;
  p.br = br;
  p.b1 = b1;
  p.b2 = b2;
  p.w1 = static_cast<const uint8_t*>(W1.data);
  p.w2 = static_cast<const uint8_t*>(W2.data);
  p.s1 = W1.scales;
  p.s2 = W2.scales;
  p.logits = logits;
  p.h = h;
  p.o = o;
  p.y = y;
  p.header = static_cast<unsigned*>(ws);
  // rows 64 bytes off a multiple of 128: two rows' 64-byte pieces on distinct banks
  p.row_pitch = (d.D > d.I ? d.D : d.I) * 2 + 64;
  p.act = act_of(d);
  if (d.wfmt == MOE_W_BF16)
    return d.T <= 8 ? launch<MOE_W_BF16, 1>(p, s) : launch<MOE_W_BF16, 2>(p, s);
  return d.T <= 8 ? launch<MOE_W_MXFP4, 1>(p, s) : launch<MOE_W_MXFP4, 2>(p, s);
}

}  // namespace moe

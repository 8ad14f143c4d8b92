// Block-scaled FP8 matrix product, dense or grouped by expert:
//
//   out[r, n] = sum_b a_scale[r, b] * w_scale[e, n / 128, b] *
//               (sum of a[r, k] * w[e, n, k] over the 128 k of block b) + bias[e, n]
//
// for the rows r of expert e's segment, a and w in E4M3. The scales vary with
// the block of the reduction, so a block's products are summed by the tensor
// cores (tcgen05 kind::f8f6f4, fp32 in TMEM) and added to the running sum with
// its scale by ordinary fp32 FMAs, out of TMEM into registers: one FMA per
// output element and block. At 8192 x 5760 x 2880 the tensor core alone needs 98
// to 107 us, reading the sums out of TMEM 98 (108 with their FMAs), the operands'
// way out of L2 96; tensor core and sums, which share TMEM, 131, all together,
// handed over block by block through two TMEM buffers, 140 (1.9 PFLOP/s in a
// burst; 168 us under the power cap). A buffer's round -- products, commit, wait,
// read, release, wait -- bounds it: the hand-overs of a block alone take some 1000
// cycles, the read 400, the products 512. Few rows: 256 on 28 of 32 experts of
// 2880 x 2880 take 48 us (4.8 TB/s; 56 with cold caches), 17 x 5760 x 2880 11 us. All
// of a tile's 128 rows are multiplied, summed and kept room for in the ring, however
// few there are, and 90 SMs have a tile of 64 of 5760 columns.
//
// Measured and not kept: halves of a tile handed over separately (157 us against
// 145), CTA pairs (291 us: both hand-overs of every block then cross CTAs),
// sixteen warps of 64 columns for the sums (181 us against 160), reads of 32
// columns whose FMAs overlap the next (160 against 140: every read waits some 200
// cycles).
//
// One persistent block per SM over tiles of 128 rows x kBN columns:
//   warps 0, 3  TMA producers of the tile's 128 x 128 block of a (a box of 32
//               rows where the tile has no more) and kBN x 128 block of w;
//   warps 1, 2  issue the four K = 32 MMAs of the even and the odd blocks (the
//               commits after every block hold an issuer up, so two take turns;
//               each always meets the same ring slots and TMEM buffers, both
//               even in number); warp 1 allocates TMEM;
//   from 4 on   a thread per row and 64 or 128 columns: keeps the running sums in
//               registers and writes the output.
// Tiles are numbered expert by expert, column tile, then row tile, from the
// offsets on the device, as in the bf16 GEMM. All waits are bounded; on a
// timeout the kernel records it, drains what is in flight and returns.
#include <algorithm>

#include "common.cuh"
#include "gemm_common.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int BM = 128;
constexpr int BK = 128;               // one scale block, one 128-byte swizzle row of E4M3
constexpr int kSmallRows = 32;        // box of a for tiles with at most this many rows
constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 8;
constexpr int kABytes = BM * BK;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kCtrlBytes = 512;
// The scales reach the threads through shared memory, kScaleBlocks blocks of K
// of a warp's 32 rows and of its columns at a time, double-buffered (a load per
// thread and block would touch 32 lines each time, and be waited for). Rows 9
// words apart: no bank conflict.
constexpr int kScaleBlocks = 8, kScalePitch = kScaleBlocks + 1, kScaleRows = 33;
constexpr int kScaleBytes = 2 * kScaleRows * kScalePitch * 4;  // per warp
constexpr size_t kMaxSmem = 232448;

struct Fp8Params {
  int R, E, N, K, KB, NB, NT;  // blocks of K, blocks of N, column tiles
  int stages;
  int out_f32;
  const float* a_scale;
  const float* w_scale;
  const int32_t* offsets;
  const uint16_t* bias;
  void* out;
  int* status;
};

// kind::f8f6f4, A = B = E4M3, D = fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A * B^T over K = 32, by a whole warp with one lane elected to
// issue (the operands stay warp-uniform, which keeps the issue short).
__device__ __forceinline__ void mma_f8_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, q;\n\t.reg .b32 r;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, q;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// mbar_wait_bounded that looks at the clock only now and then: the waits of this
// pipeline mostly last less than a reading of it.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 63u) == 0) {
      if (abort && *abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitNs) return false;
    }
  }
  return true;
}

// c0 += s * v0, c1 += s * v1 in one instruction.
__device__ __forceinline__ void fma2(float& c0, float& c1, float s, uint32_t v0, uint32_t v1) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%3, %4};\n\t"
      "mov.b64 b, {%2, %2};\n\t"
      "mov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "+f"(c0), "+f"(c1)
      : "f"(s), "r"(v0), "r"(v1));
}

// 32 lanes x 64 consecutive 32-bit columns per thread, waited for (in one
// statement, so that no use of them can come before the wait).
__device__ __forceinline__ void tmem_ld_x64(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
        "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
        "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
        "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
        "=r"(v[30]), "=r"(v[31]), "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]),
        "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]), "=r"(v[41]),
        "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
        "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]),
        "=r"(v[54]), "=r"(v[55]), "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]),
        "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr)
      : "memory");
}

// A tile's columns and the warps that hold its sums, and what follows.
template <int kBN_, int kSumWarps_>
struct Shape {
  static constexpr int kBN = kBN_, kSumWarps = kSumWarps_;
  static constexpr int kThreads = 128 + 32 * kSumWarps;
  static constexpr int kCols = kBN / (kSumWarps / 4);  // columns per thread
  static constexpr int kBufs = kMaxBufs * kBN <= 512 ? kMaxBufs : 512 / kBN / 2 * 2;  // TMEM buffers, even
  static constexpr uint32_t kTmemCols = kBufs * kBN <= 256 ? 256 : 512;
  static constexpr uint32_t kStageBytes = kABytes + kBN * BK;
  // Registers per thread of the four control warps and of the others, out of
  // what the launch gets (a multiple of 8 per thread); four warps of sums have
  // enough as it is.
  static constexpr bool kMoveRegs = kSumWarps > 4;
  static constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
  static constexpr int kRegsControl = 56;
  static constexpr int kRegsSums = (kRegsLaunch * kThreads - 128 * kRegsControl) / (32 * kSumWarps) / 8 * 8;
  static_assert(!kMoveRegs || (kRegsSums > kRegsLaunch && kRegsSums <= 232), "");
  static_assert(kCols % 64 == 0 && 128 % kCols == 0, "");
};

template <class S_>
__global__ void __launch_bounds__(S_::kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                    const __grid_constant__ CUtensorMap tmB, const Fp8Params p) {
  constexpr int kBN = S_::kBN, kCols = S_::kCols, kBufs = S_::kBufs, kSumWarps = S_::kSumWarps;
  constexpr uint32_t kTmemCols = S_::kTmemCols, kStageBytes = S_::kStageBytes;
  constexpr int kRegsControl = S_::kRegsControl, kRegsSums = S_::kRegsSums;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  float* scales = reinterpret_cast<float*>(smem + S * kStageBytes);
  uint8_t* ctrl = smem + S * kStageBytes + kSumWarps * kScaleBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ctrl);  // full[8] empty[8] tfull[8] tempty[8] done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (2 * kMaxStages + 2 * kMaxBufs + 1));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* bad_s = reinterpret_cast<int*>(tmem_slot + 2);
  int* seg = reinterpret_cast<int*>(ctrl + kCtrlBytes);  // E+1 segment starts
  int* tpre = seg + (p.E + 1);                           // E+1 tile prefix

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kMaxStages + kMaxBufs + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * kMaxStages + 2 * kMaxBufs);

  // ---- prologue: segment table, tile prefix, barriers, TMEM
  if (threadIdx.x == 0) {
    *bad_s = 0;
    *abort_flag = 0;
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
    const int o = p.offsets ? p.offsets[e] : e * p.R;
    seg[e] = o;
    if (o < 0 || o > p.R || (e == 0 && o != 0)) atomicOr(bad_s, 1);
  }
  __syncthreads();
  if (warp == 0) {
    const int per = (p.E + 31) / 32;
    const int e0 = lane * per;
    int local = 0;
    for (int e = e0; e < e0 + per && e < p.E; ++e) {
      const int cnt = seg[e + 1] - seg[e];
      if (cnt < 0) atomicOr(bad_s, 1);
      local += cnt > 0 ? (cnt + BM - 1) / BM * p.NT : 0;
    }
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    int run = incl - local;
    for (int e = e0; e < e0 + per && e < p.E; ++e) {
      tpre[e] = run;
      const int cnt = seg[e + 1] - seg[e];
      run += cnt > 0 ? (cnt + BM - 1) / BM * p.NT : 0;
    }
    if (lane == 31) tpre[p.E] = incl;
    __syncwarp();
    if (lane == 0) {
      if (*bad_s) {
        record_status(p.status, MOE_ERR_DEVICE_BOUNDS);
        tpre[p.E] = 0;
      }
      for (int s = 0; s < S; ++s) {
        mbar_init(full_bar(s), 2);  // both producers
        mbar_init(empty_bar(s), 1);
      }
      for (int b = 0; b < kBufs; ++b) {
        mbar_init(tfull_bar(b), 1);
        mbar_init(tempty_bar(b), kSumWarps);
      }
      mbar_init(done_bar, 2);
      fence_mbar_init();
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmA32);
      tma_prefetch_desc(&tmB);
    }
  } else if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = tpre[p.E];

  if (warp < 4) {
    if constexpr (S_::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0 || warp == 3) {
      if (lane == 0) {
        // -------------------------------------------------------- producers
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool failed = false;
        for (int tile = blockIdx.x; tile < total && !failed; tile += gridDim.x) {
          int e, nt, mt;
          decode_tile(tile, tpre, seg, p.E, BM, e, nt, mt);
          const int row0 = seg[e] + mt * BM;
          const bool small = seg[e + 1] - row0 <= kSmallRows;
          const CUtensorMap* map = warp == 3 ? &tmB : small ? &tmA32 : &tmA;
          const uint32_t bytes = warp == 3 ? kBN * BK : small ? kSmallRows * BK : kABytes;
          const int at = warp == 3 ? e * p.N + nt * kBN : row0;
          for (int kb = 0; kb < p.KB; ++kb) {
            if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag)) {
              failed = true;
              break;
            }
            mbar_arrive_expect_tx(full_bar(stage), bytes);
            tma_load_2d(smem_u32(smem + stage * kStageBytes) + (warp == 3 ? kABytes : 0), map, full_bar(stage),
                        kb * BK, at);
            ++issued;
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (failed) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
          // let the copies still in flight land before the CTA can exit
          for (int i = issued < S ? issued : S; i > 0; --i) {
            if (--stage < 0) {
              stage = S - 1;
              phase ^= 1u;
            }
            wait_bounded(full_bar(stage), phase, nullptr);
          }
        }
      }
    } else {
      // ---------------------------------------------------------- MMA issuers
      const int mine = warp - 1;  // parity of this issuer's blocks, counted over all tiles
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0, count = 0;
      bool failed = false;
      for (int tile = blockIdx.x; tile < total && !failed; tile += gridDim.x) {
        int e, nt, mt;
        decode_tile(tile, tpre, seg, p.E, BM, e, nt, mt);
        const uint32_t idesc = idesc_e4m3_f32(BM, min(kBN, p.N - nt * kBN));
        for (int kb = 0; kb < p.KB; ++kb, ++count) {
          if (static_cast<int>(count & 1u) == mine) {
            if (!__all_sync(0xffffffffu, wait_bounded(full_bar(stage), phase, abort_flag) &&
                                             wait_bounded(tempty_bar(buf), buf_phase ^ 1u, abort_flag))) {
              failed = true;
              break;
            }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + buf * kBN;
            const uint32_t a_addr = smem_u32(smem + stage * kStageBytes);
            const uint32_t b_addr = a_addr + kABytes;
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              mma_f8_elect(d_tmem, desc_kmajor_sw128(a_addr + kk * 32), desc_kmajor_sw128(b_addr + kk * 32), idesc,
                           kk != 0 ? 1u : 0u);
            tc_commit_elect(tfull_bar(buf));
            tc_commit_elect(empty_bar(stage));
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == kBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      if (failed && lane == 0) {
        record_status(p.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // all MMAs issued by this warp complete before TMEM is released
      __syncwarp();
      tc_commit_elect(done_bar);
      wait_bounded(done_bar, 0, nullptr);
    }
  } else {
    if constexpr (S_::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
    // ------------------------------------------------- running sums and output
    const int q = warp & 3;            // TMEM lane quarter this warp may access
    const int part = (warp - 4) / 4;   // its part of the columns
    float* mine = scales + (warp - 4) * 2 * kScaleRows * kScalePitch;
    // The scales of a tile's 32 rows (past the segment's last row, that row's)
    // and of its columns: aim at a tile, then ask for blocks [kb, kb +
    // kScaleBlocks). Lanes 8 i + j bring block kb + j of rows i, i + 4, ...
    const int sj = lane % kScaleBlocks, sr = lane / kScaleBlocks;
    const float *sa = nullptr, *sw = nullptr;
    int s_last = 0;  // the last of the 32 rows that may be read
    auto aim = [&](int e, int nt, int mt) {
      const int first = seg[e] + mt * BM + q * 32, last = seg[e + 1] - 1;
      const int nb = min((nt * kBN + part * kCols) / 128, p.NB - 1);
      s_last = last - first;
      sa = p.a_scale + static_cast<int64_t>(first) * p.KB + sj;
      sw = p.w_scale + (static_cast<int64_t>(e) * p.NB + nb) * p.KB + sj;
    };
    auto ask = [&](int kb, int b) {
      const uint32_t to = smem_u32(mine + b * kScaleRows * kScalePitch + sr * kScalePitch + sj);
      if (kb + sj < p.KB) {
        if (s_last >= 31) {
          const float* from = sa + sr * p.KB + kb;
#pragma unroll
          for (int i = 0; i < kScaleBlocks; ++i, from += 4 * p.KB) cp_async4(to + i * (4 * kScalePitch * 4), from);
        } else {
#pragma unroll 1
          for (int i = 0; i < kScaleBlocks; ++i)
            cp_async4(to + i * (4 * kScalePitch * 4), sa + static_cast<int64_t>(min(i * 4 + sr, s_last)) * p.KB + kb);
        }
        if (sr == 0) cp_async4(to + 32 * kScalePitch * 4, sw + kb);
      }
      cp_async_commit();
    };
    int buf = 0, sbuf = 0;
    uint32_t buf_phase = 0;
    bool failed = false;
    const uint32_t from = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + part * kCols;
    int e = 0, nt = 0, mt = 0;
    if (blockIdx.x < total) {
      decode_tile(blockIdx.x, tpre, seg, p.E, BM, e, nt, mt);
      aim(e, nt, mt);
      ask(0, 0);
    }
    for (int tile = blockIdx.x; tile < total && !failed; tile += gridDim.x) {
      const int row = seg[e] + mt * BM + q * 32 + lane;
      const bool valid = row < seg[e + 1];
      const int n0 = nt * kBN + part * kCols;
      const int this_e = e;
      const bool more = tile + static_cast<int>(gridDim.x) < total;
      if (more) decode_tile(tile + gridDim.x, tpre, seg, p.E, BM, e, nt, mt);
      // the sums start at the bias, which arrives while the first block is multiplied
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 8) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (p.bias && n0 + c < p.N)  // (N is a multiple of 16)
          unpack8(__ldg(reinterpret_cast<const uint4*>(p.bias + static_cast<int64_t>(this_e) * p.N + n0 + c)), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c + i] = f[i];
      }
      for (int kb = 0; kb < p.KB; ++kb) {
        if (kb % kScaleBlocks == 0) {
          // the following blocks' scales, the next tile's first after the last
          if (kb + kScaleBlocks < p.KB)
            ask(kb + kScaleBlocks, sbuf ^ 1);
          else if (more) {
            aim(e, nt, mt);
            ask(0, sbuf ^ 1);
          } else
            cp_async_commit();
          cp_async_wait_1();
          __syncwarp();
          sbuf ^= 1;
        }
        const float* at = mine + (sbuf ^ 1) * kScaleRows * kScalePitch + kb % kScaleBlocks;
        const float s = at[lane * kScalePitch] * at[32 * kScalePitch];
        if (!__all_sync(0xffffffffu, wait_bounded(tfull_bar(buf), buf_phase, abort_flag))) {
          failed = true;
          break;
        }
        tc_fence_after();
        uint32_t v[64];
#pragma unroll
        for (int c = 0; c < kCols; c += 64) {
          tmem_ld_x64(from + buf * kBN + c, v);
          if (c + 64 == kCols) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(buf));
          }
#pragma unroll
          for (int i = 0; i < 64; i += 2) fma2(acc[c + i], acc[c + i + 1], s, v[i], v[i + 1]);
        }
        if (++buf == kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (failed) {
        if (lane == 0) {
          record_status(p.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        break;
      }
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        if (n0 + c >= p.N) break;  // (uniform; N is a multiple of 16)
        if (!valid) continue;
        const int64_t at = static_cast<int64_t>(row) * p.N + n0 + c;
        if (p.out_f32) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[c + i];
          st_global_v8f(static_cast<float*>(p.out) + at, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[c + 8 + i];
          st_global_v8f(static_cast<float*>(p.out) + at + 8, v);
        } else {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = pack_bf16x2(acc[c + 2 * i], acc[c + 2 * i + 1]);
          st_global_v8u(static_cast<uint16_t*>(p.out) + at, v);
        }
      }
    }
  }

  asm volatile("cp.async.wait_all;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// 2-D tensor of `rows` rows of `inner` bytes, loaded in boxes of 128 bytes x
// box_rows rows with the 128-byte swizzle; elements outside read as zero.
bool make_tmap_u8(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows) {
  auto fn = tma_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {inner};
  cuuint32_t box[2] = {BK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class S_>
moe_status_t launch(Fp8Params p, const uint8_t* a, const uint8_t* w, cudaStream_t s) {
  CUtensorMap ta, ta32, tb;
  if (!make_tmap_u8(&ta, a, p.K, p.R, BM) || !make_tmap_u8(&ta32, a, p.K, p.R, kSmallRows) ||
      !make_tmap_u8(&tb, w, p.K, static_cast<uint64_t>(p.E) * p.N, S_::kBN))
    return MOE_ERR_CUDA;
  constexpr size_t stage = S_::kStageBytes;
  const size_t fixed = 1024 + kCtrlBytes + S_::kSumWarps * kScaleBytes + 2 * (p.E + 1) * sizeof(int);
  p.stages = static_cast<int>((kMaxSmem - fixed) / stage);
  p.stages = p.stages > kMaxStages ? kMaxStages : p.stages / 2 * 2;
  p.NT = (p.N + S_::kBN - 1) / S_::kBN;
  const size_t smem = fixed + p.stages * stage;
  // (the same limit for every size: calls from several host threads do not meet another's)
  if (cudaFuncSetAttribute(fp8_gemm_kernel<S_>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kMaxSmem)) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int64_t max_tiles = ((p.R + BM - 1) / BM + p.E) * static_cast<int64_t>(p.NT);
  const int grid = static_cast<int>(max_tiles < num_sms() ? max_tiles : num_sms());
  fp8_gemm_kernel<S_><<<grid, S_::kThreads, smem, s>>>(ta, ta32, tb, p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

moe_status_t launch_fp8_matmul(const moe_fp8_t& d, const uint8_t* a, const float* a_scale, const int32_t* offsets,
                               const uint8_t* w, const float* w_scale, const uint16_t* bias, void* out, int* status,
                               cudaStream_t s) {
  Fp8Params p{};
  p.R = d.R;
  p.E = d.E;
  p.N = d.N;
  p.K = d.K;
  p.KB = (d.K + 127) / 128;
  p.NB = (d.N + 127) / 128;
  p.out_f32 = d.out_type == MOE_T_F32;
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.offsets = offsets;
  p.bias = bias;
  p.out = out;
  p.status = status;
  // The tile whose rounds over the SMs cost least: a block of K takes 0.62 us at
  // 256 columns (0.66 where tiles have few rows and the weights' stream sets the
  // time), 0.54 at 192, 0.29 at 64. Rounds are whole ones for a dense product; for
  // several experts, whose rows the host does not know, they are estimated, with
  // half a round for the tail. Measured in us at 256 / 192 / 64 columns, a launch
  // among others on operands that the L2 has not, on both sides of the borders.
  // 5760 columns, K = 2880: 128 rows 16.8 / 16.0 / 11.5, 200 rows 17.1 / 16.0 / 18.5,
  // 1024 rows 30.3 / 27.2 / 37.6, 1536 rows 30.4 / 38.9 / 56.6, 8192 rows 147 / 162 /
  // 264. 32 experts (28 with rows) of 2880 x 2880: 256 rows 53.5 / 48.3 / 69.8, 4096
  // rows 69.2 / 74.7 / 107; 8 of 4096 x 4096: 8 rows 22.8 / 22.2 / 26.6, 256 rows 27.8
  // / 39.4 / 41.8. Over 120 sizes, up to 16384 rows and 128 experts, the chosen tile
  // takes 0.6% more than the best on average, 16% at worst.
  const bool few = d.R < 64LL * d.E;
  const int64_t mtiles = d.E == 1 ? (d.R + 127) / 128 : few ? std::min(d.E, d.R) : d.R / 128 + d.E;
  auto cost = [&](int bn, double us) {
    const int64_t tiles = mtiles * ((d.N + bn - 1) / bn);
    if (d.E == 1) return us * static_cast<double>((tiles + num_sms() - 1) / num_sms());
    return us * std::max(1.0, static_cast<double>(tiles) / num_sms() + 0.5);
  };
  const double c256 = cost(256, few ? 0.66 : 0.62), c192 = cost(192, 0.54), c64 = cost(64, 0.29);
  if (c64 <= c192 && c64 <= c256) return launch<Shape<64, 4>>(p, a, w, s);
  if (c192 <= c256) return launch<Shape<192, 12>>(p, a, w, s);
  return launch<Shape<256, 8>>(p, a, w, s);
}

}  // namespace moe

// Block-scaled fp8 products for many rows on the 5th-generation tensor cores
// (tcgen05 + TMEM, TMA), dense or grouped by expert:
//
//   out[m][n] = sum_kb sa[m][kb] sw[n / 128][kb] (sum_{k in block kb} a[m][k] w[n][k])
//
// mode 0 (gate/up): two such products over the same rows, h = silu(gate) * up, and h
// quantised like every activation row: hs = max(max |h| / 448, 2^-126) per 128 columns,
// code = e4m3(h * (1 / hs)).  mode 1: the product, stored as f32 or bf16.
//
// The scales differ from block to block of K, so the tensor cores may only sum inside one
// block: every 128 of K the accumulators leave TMEM and are added, scaled, to fp32 sums in
// registers.  A thread owns one row, so the factor sa * sw is one number for all its columns.
//
// One persistent kernel, one CTA per SM, 128 x 256 tiles:
//   warp 0      TMA producer: per 128 of K, A 128 rows and 256 weight rows, 128-byte swizzle, 4
//               stages of 48 KB.  (Gathering the pairs' token rows here, four per TMA load,
//               took twice the time of the products: 32 loads to issue per stage instead of
//               one.  fp8_gather_kernel copies them first.)
//   warp 1      MMA issuer: tcgen05.mma kind::f8f6f4, M=128, N=256, K=32, into two TMEM buffers
//               of 256 columns in turn, so the tensor cores fill one while the other is read.
//   warps 2, 3  factors: sa * sw of every row for 8 blocks of K at a time, into shared memory.
//               (Read from global memory by the summing threads, the row scales' 32 separate
//               lines per warp cost half of their time.)
//   warps 4-11  sums: warp w reads TMEM lanes 32 (w % 4).. of one half of the columns, adds
//               them to 128 sums per thread, and at the end of a tile stores them.  These warps
//               take 224 registers each from the 168 of the launch, the other four keep 56.  The
//               loop must not spill: the reloads miss the small L1 beside the ring (8 bytes of
//               spill cost 10 % of the kernel).
//
// What bounds it: 8192 x 7168 x 4096 takes 240 to 244 us, 2.0 PFLOP/s, a hundred times in a row, and
// 283 us, 1.7 PFLOP/s, over seconds, when the power cap lowers the clock (cuBLAS reaches 3.3 at 8192^3 in
// short runs with one scale per tensor, that is, without leaving TMEM).  The tensor cores alone would take 515 cycles
// per block of K (616 with the loads running); the loop takes about 850, because a TMEM buffer is
// free only after release -> issue (200) -> its MMAs and commit (700 to 800) -> loads and
// three quarters of the multiply-adds (600), and two buffers of 256 columns fill TMEM.  Tried and
// slower: halves of N = 128 with two buffers each (the shared-memory reads of A double), 16
// summing warps (spills), two CTAs per SM with 128 x 128 tiles, paired multiply-adds (moves).
//
// gate/up tiles hold 128 gate and 128 up columns; each half of the warps takes 64 columns of
// both, so silu(gate) * up stays inside a thread.
//
// Every wait is bounded: a thread that gives up records 121-125 in *err and raises the CTA's
// abort flag; all roles then leave, with their copies and MMAs landed, and TMEM is released.
#include "fp8.hpp"
#include "fp8_common.cuh"
#include "fp8_mma.cuh"

namespace ftk {
namespace {

constexpr int BM = 128, BN = 256, BK = kFp8Block;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 4, TMEM_COLS = 512;
constexpr int SUM_WARPS = 8, THREADS = 128 + 32 * SUM_WARPS;
constexpr int HN = BN / 2;    // columns of a summing thread: half of the tile's
constexpr int LC = 32;        // columns of a TMEM load
constexpr int FK = 8;         // blocks of K per chunk of factors
// registers: (4 * 56 + 8 * 224) * 32 = 384 * 168, the launch's
constexpr int CONTROL_REGS = 56, SUM_REGS = 224;

struct Smem {
  uint64_t full[STAGES], done[STAGES], tempty[2], ffull[2], fempty[2], halves, never;
  uint32_t tmem_base;
  int abort;
  int mt_start[kMaxList + 1];   // prefix of M-tiles over the groups
  int row_start[kMaxList];
  int rows[kMaxList];
  float amax[2][2][BM];         // gate/up: a row's largest |h| per half, double-buffered by tile
  float factor[2][FK][2][BM];   // sa * sw of a row: by half of the columns, or for gate and up
};

// Eight words to a 32-byte aligned address, or a 16-byte aligned one.
FT_DEVICE void st_row(void* p, const uint32_t (&w)[8], bool sector) {
  if (sector) {
    st_sector(p, w);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// v[i] of lane l <-> v[l] of lane i.
FT_DEVICE void transpose32(uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(i & o)) {   // trade v[i] of the upper lane for v[i + o] of the lower
        const uint32_t give = up ? v[i] : v[i + o];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, o);
        if (up) v[i] = got; else v[i + o] = got;
      }
  }
}

template <int MODE>
__global__ void __launch_bounds__(THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ GemmGroups groups,
                const __grid_constant__ Fp8Gemm p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Smem* S = reinterpret_cast<Smem*>(base + STAGES * STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (p.K + BK - 1) / BK;
  constexpr int TN = MODE == 0 ? BN / 2 : BN;   // output columns of a tile
  const int n_tiles = (p.N + TN - 1) / TN;
  int* err = p.err;

  for (int g = threadIdx.x; g < groups.n; g += THREADS) {
    const int e = groups.expert[g];
    const int r0 = e >= 0 ? p.offsets[e] : p.T * p.k;
    S->row_start[g] = r0;
    S->rows[g] = e >= 0 ? p.offsets[e + 1] - r0 : p.T;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&S->full[s], 1);
      mbar_init(&S->done[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S->tempty[b], SUM_WARPS);
      mbar_init(&S->ffull[b], 2);
      mbar_init(&S->fempty[b], SUM_WARPS);
    }
    mbar_init(&S->halves, SUM_WARPS);
    mbar_init(&S->never, 1);
    S->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&S->tmem_base)), "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncthreads();
  if (warp == 0) {   // prefix sum of the groups' M-tiles
    int acc = 0;
    for (int g0 = 0; g0 < groups.n; g0 += 32) {
      const int g = g0 + lane;
      int v = g < groups.n ? (S->rows[g] + BM - 1) / BM : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      if (g < groups.n) S->mt_start[g + 1] = acc + v;
      acc += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) S->mt_start[0] = 0;
  }
  fp8_fence_before();
  __syncthreads();
  fp8_fence_after();
  const uint32_t tmem = S->tmem_base;
  const int total_tiles = S->mt_start[groups.n] * n_tiles;   // times 2^15 outputs: far below 2^31
  volatile int* abort_flag = &S->abort;

  // tile -> (group, m-tile, n-tile): the M-tiles that share a weight tile run back to back
  auto decode = [&](int t, int& g, int& m, int& n) {
    int lo = 0, hi = groups.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (S->mt_start[mid] * n_tiles <= t) lo = mid; else hi = mid - 1;
    }
    g = lo;
    const int local = t - S->mt_start[g] * n_tiles;
    const int mtg = S->mt_start[g + 1] - S->mt_start[g];
    n = local / mtg;
    m = local - n * mtg;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CONTROL_REGS));
    if (warp == 0) {   // ------------------------------------------------ TMA producer
      int it = 0;
      for (int t = blockIdx.x; t < total_tiles && !*abort_flag; t += gridDim.x) {
        if (t == (int)blockIdx.x + p.fail_at * (int)gridDim.x) {
          never_wait(&S->never, abort_flag, err, 121);
          break;
        }
        int g, m, n;
        decode(t, g, m, n);
        const int row0 = S->row_start[g] + m * BM, z = groups.z[g];
        bool stop = false;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int s = it % STAGES;
          if (!warp_wait(&S->done[s], ((it / STAGES) & 1) ^ 1, abort_flag, err, 121)) {
            stop = true;
            break;
          }
          if (elect_one()) {
            unsigned char* sa = base + s * STAGE_BYTES;
            unsigned char* sb = sa + A_BYTES;
            mbar_expect_tx(&S->full[s], STAGE_BYTES);
            fp8_tma_2d(sa, &maps.a, &S->full[s], kb * BK, row0);
            fp8_tma_3d(sb, &maps.b[0], &S->full[s], kb * BK, n * TN, z);
            fp8_tma_3d(sb + B_BYTES / 2, &maps.b[1], &S->full[s], kb * BK, MODE == 0 ? n * TN : n * TN + BN / 2, z);
          }
          __syncwarp();
        }
        if (stop) break;
      }
      // drain: wait (bounded) until every issued stage has landed
      if (lane == 0)
        for (int j = it - STAGES < 0 ? 0 : it - STAGES; j < it; ++j) mbar_drain(&S->full[j % STAGES], (j / STAGES) & 1);
    } else if (warp == 1) {   // ------------------------------------------- MMA issuer
      constexpr uint32_t idesc = fp8_idesc(BM, BN);
      const uint64_t desc0 = fp8_desc(smem_u32(base));   // stage s, K step kk: + (s * STAGE_BYTES + kk * 32) / 16
      // a block starts its sums afresh: the issuer sees blocks, not tiles
      const int mine = total_tiles > (int)blockIdx.x ? (total_tiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
      int it = 0;
      for (long long left = (long long)mine * KB; left > 0; --left, ++it) {
        const int s = it % STAGES, b = it & 1;
        if (!warp_wait2(&S->full[s], (it / STAGES) & 1, &S->tempty[b], ((it >> 1) & 1) ^ 1, abort_flag, err, 122))
          break;
        fp8_fence_after();
        if (elect_one()) {
          const uint64_t da = desc0 + (uint32_t)(s * (STAGE_BYTES >> 4)), db = da + (A_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk) fp8_mma(tmem + b * BN, da + 2 * kk, db + 2 * kk, idesc, kk ? 1u : 0u);
          fp8_commit(&S->done[s]);   // frees the stage and hands the buffer to the sums
        }
        __syncwarp();
      }
      // drain: the last commit stands for every MMA issued (the sums may have given up on them)
      if (lane == 0 && it > 0) mbar_drain(&S->done[(it - 1) % STAGES], ((it - 1) / STAGES) & 1);
    } else {   // ---------------------------------------------------------- factors
      const int r0 = threadIdx.x - 64;   // rows r0 and r0 + 64 of the tile
      const int NB = (p.N + kFp8Block - 1) / kFp8Block;
      int ch = 0;
      for (int t = blockIdx.x; t < total_tiles && !*abort_flag; t += gridDim.x) {
        int g, m, n;
        decode(t, g, m, n);
        const int first = S->row_start[g], last = first + S->rows[g] - 1;
        const float* sa[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // rows past the group repeat its last
          int row = min(first + m * BM + r0 + 64 * i, last);
          if (MODE == 0) row = groups.expert[g] < 0 ? row - p.T * p.k : p.perm[row] / p.k;
          sa[i] = p.a_scales + (long long)row * KB;
        }
        // weight scales: gate and up of the tile's block of I, or the blocks of the tile's two halves
        const long long wz = groups.z[g] * p.blob;
        const float* sw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int nb = MODE == 0 ? n : min(2 * n + i, NB - 1);
          sw[i] = reinterpret_cast<const float*>(p.w_scales[i] + wz) + (long long)nb * KB;
        }
        bool ok = true;
        for (int k0 = 0; k0 < KB; k0 += FK, ++ch) {
          const int b = ch & 1;
          ok = warp_wait(&S->fempty[b], ((ch >> 1) & 1) ^ 1, abort_flag, err, 125);
          if (!ok) break;
#pragma unroll 1
          for (int j0 = 0; j0 < FK; j0 += 4) {   // four blocks at a time: these warps have few registers
            float w[2][4], a[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int kb = min(k0 + j0 + j, KB - 1);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                w[i][j] = sw[i][kb];
                a[i][j] = sa[i][kb];
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                S->factor[b][j0 + j][0][r0 + 64 * i] = a[i][j] * w[0][j];
                S->factor[b][j0 + j][1][r0 + 64 * i] = a[i][j] * w[1][j];
              }
          }
          warp_arrive(&S->ffull[b]);
        }
        if (!ok) break;
      }
    }
  } else {   // -------------------------------------------------------- sums and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SUM_REGS));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r = q * 32 + lane;               // tile row of this thread
    const int NB = (p.N + kFp8Block - 1) / kFp8Block;
    constexpr int NL = HN / LC;                // TMEM loads per block
    // half h sums columns 128 h .. of a product tile; columns 64 h .. of gate and of up
    const uint32_t col0 = tmem + ((uint32_t)(q * 32) << 16) + half * (MODE == 0 ? HN / 2 : HN);
    auto column = [&](int c) {
      return MODE == 0 ? (c / (NL / 2)) * (BN / 2) + (c % (NL / 2)) * LC : c * LC;
    };
    int it = 0, tl = 0, ch = 0;
    for (int t = blockIdx.x; t < total_tiles && !*abort_flag; t += gridDim.x, ++tl) {
      float acc[HN];
#pragma unroll
      for (int i = 0; i < HN; ++i) acc[i] = 0.f;
      // The next columns are asked for before these are added, the next block's first before
      // this one's last, so that the wait for the tensor cores and the load's latency pass behind
      // multiply-adds.  No load is pending where the loop turns (tmem_wait).
      uint32_t v[2][LC];
      auto ready = [&](int i) {   // accumulators of block i (over the tiles)
        const bool w = warp_wait(&S->done[i % STAGES], (i / STAGES) & 1, abort_flag, err, 123);
        fp8_fence_after();
        return w;
      };
      bool ok = ready(it);
      if (!ok) break;
      tmem_ld(col0 + (it & 1) * BN, v[0]);
      tmem_wait(v[0]);
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const int b = it & 1, j = kb % FK, fb = ch & 1;
        if (j == 0) {
          ok = warp_wait(&S->ffull[fb], (ch >> 1) & 1, abort_flag, err, 123);
          if (!ok) break;
        }
        const uint32_t ta = col0 + b * BN;
        const float f0 = S->factor[fb][j][MODE == 0 ? 0 : half][r], f1 = MODE == 0 ? S->factor[fb][j][1][r] : f0;
#pragma unroll
        for (int c = 0; c < NL; ++c) {
          if (c + 1 < NL) {
            tmem_ld(ta + column(c + 1), v[(c + 1) & 1]);
          } else {
            fp8_fence_before();
            if (lane == 0) mbar_arrive(&S->tempty[b]);   // the loads were the whole warp's: all have landed
            const bool chunk_done = j == FK - 1 || kb == KB - 1;
            if (chunk_done) warp_arrive(&S->fempty[fb]);
            ch += chunk_done;
            if (kb + 1 < KB) {
              ok = ready(it + 1);
              if (!ok) break;
              tmem_ld(col0 + (b ^ 1) * BN, v[0]);
            }
          }
#pragma unroll
          for (int i = 0; i < LC; ++i) fma_col(acc[LC * c + i], v[c & 1][i], MODE == 0 && c >= NL / 2 ? f1 : f0);
          tmem_wait(v[(c + 1) & 1]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      int g, m, n;   // not before: the loop has no register to spare for them
      decode(t, g, m, n);
      const bool valid = r < S->rows[g] - m * BM;
      const long long row = S->row_start[g] + (long long)m * BM + r;
      if (MODE == 0) {
        constexpr int HC = HN / 2;   // h columns of this half
        float h[HC], mx = 0.f;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          h[i] = silu_fast(acc[i]) * acc[HC + i];
          mx = amax_nan(mx, h[i]);
        }
        S->amax[tl & 1][half][r] = mx;
        warp_arrive(&S->halves);
        ok = warp_wait(&S->halves, tl & 1, abort_flag, err, 124);
        if (!ok) break;
        mx = amax_nan(mx, S->amax[tl & 1][half ^ 1][r]);
        const float sc = fp8_scale(mx), inv = 1.0f / sc;
        if (valid) {
          const int c0 = n * TN + half * HC;
          uint8_t* dst = static_cast<uint8_t*>(p.out) + row * p.N + c0;
#pragma unroll
          for (int j = 0; j < HC / 16; ++j)
            if (c0 + 16 * j < p.N) {   // N is a multiple of 16
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float* v = h + 16 * j + 4 * i;
                w[i] = e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16;
              }
              *reinterpret_cast<uint4*>(dst + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          if (half == 0) p.out_scales[row * NB + n] = sc;
        }
      } else {
        const int c0 = n * TN + half * HN;
        const int es = p.out_bf16 ? 2 : 4;
        unsigned char* dst = static_cast<unsigned char*>(p.out) + (row * p.ldo + c0) * es;
        if (((p.ldo * es) & 15) == 0 && ((uintptr_t)p.out & 15) == 0) {
          // a thread stores its own row, a 32-byte sector at a time (two halves where rows are
          // 16-byte aligned only)
          const bool sectors = ((p.ldo * es) & 31) == 0 && ((uintptr_t)p.out & 31) == 0;
          if (valid) {
            if (p.out_bf16) {
#pragma unroll
              for (int j = 0; j < HN / 16; ++j) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = bf16x2(acc[16 * j + 2 * i], acc[16 * j + 2 * i + 1]);
                if (c0 + 16 * j + 16 <= p.N) {
                  st_row(dst + 32 * j, w, sectors);
                } else {
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    if (c0 + 16 * j + i < p.N)
                      reinterpret_cast<uint16_t*>(dst)[16 * j + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                }
              }
            } else {
#pragma unroll
              for (int j = 0; j < HN / 8; ++j) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(acc[8 * j + i]);
                if (c0 + 8 * j + 8 <= p.N) {
                  st_row(dst + 32 * j, w, sectors);
                } else {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (c0 + 8 * j + i < p.N) reinterpret_cast<uint32_t*>(dst)[8 * j + i] = w[i];
                }
              }
            }
          }
        } else {
          // any other row: the warp transposes 32 x 32 values, so that its lanes store 32
          // consecutive columns of a row
          const int rows_left = S->rows[g] - m * BM - q * 32;
#pragma unroll
          for (int j = 0; j < HN / 32; ++j) {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[32 * j + i]);
            transpose32(v, lane);
            const int col = c0 + 32 * j + lane;
            if (col < p.N) {
              const long long at = (row - lane) * p.ldo + col;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < rows_left) {
                  if (p.out_bf16)
                    static_cast<uint16_t*>(p.out)[at + i * p.ldo] = (uint16_t)bf16x2(__uint_as_float(v[i]), 0.f);
                  else
                    static_cast<uint32_t*>(p.out)[at + i * p.ldo] = v[i];
                }
            }
          }
        }
      }
      __syncwarp();
    }
  }
  fp8_fence_before();
  __syncthreads();
  fp8_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

// The token row of every listed pair, H bytes (a multiple of 16) at dst + pair * stride.
// One warp per row; bound by memory (the reads hit the L2).
__global__ void __launch_bounds__(256)
fp8_gather_kernel(const uint8_t* x, long long ldx, const __grid_constant__ GemmGroups groups, const int* offsets,
                  const int* perm, int T, int k, int H, uint8_t* dst, long long stride) {
  const int g = blockIdx.y, e = groups.expert[g], lane = threadIdx.x & 31;
  const int first = e >= 0 ? offsets[e] : T * k, last = e >= 0 ? offsets[e + 1] : T * k + T;
  for (int q = first + blockIdx.x * 8 + (threadIdx.x >> 5); q < last; q += gridDim.x * 8) {
    const int tok = e >= 0 ? perm[q] / k : q - T * k;
    const uint4* from = reinterpret_cast<const uint4*>(x + tok * ldx);
    uint4* to = reinterpret_cast<uint4*>(dst + q * stride);
    const int n = H / 16;
    for (int i = lane; i < n; i += 128) {   // four loads in flight per lane
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + 32 * j < n) v[j] = from[i + 32 * j];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + 32 * j < n) to[i + 32 * j] = v[j];
    }
  }
}

constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + sizeof(Smem);

template <int MODE>
cudaError_t launch_mode(const Fp8Maps& maps, const GemmGroups& groups, const Fp8Gemm& p, int grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  fp8_gemm_kernel<MODE><<<grid, THREADS, kSmemBytes, s>>>(maps, groups, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_gemm(int mode, const Fp8Maps& maps, const GemmGroups& groups, const Fp8Gemm& p, int num_sms,
                            cudaStream_t s) {
  if (groups.n <= 0 || p.T <= 0 || p.N <= 0) return cudaSuccess;
  // an upper bound of the tile count (the groups' sizes are on the device); CTAs beyond the
  // real count leave at once
  const int tn = mode == 0 ? BN / 2 : BN;
  const long long tiles = (((long long)p.T * p.k + p.T + BM - 1) / BM + groups.n) * ((p.N + tn - 1) / tn);
  const int grid = (int)(tiles < num_sms ? tiles : num_sms);
  return mode == 0 ? launch_mode<0>(maps, groups, p, grid, s) : launch_mode<1>(maps, groups, p, grid, s);
}

cudaError_t launch_fp8_gather(const void* x, long long ldx, const GemmGroups& groups, const int* offsets,
                              const int* perm, int T, int k, int H, void* dst, long long stride, cudaStream_t s) {
  if (groups.n <= 0 || T <= 0) return cudaSuccess;
  // 32 rows per block, and blocks for the rows that a group can have: those past its rows leave at
  // once (few blocks per group made the shared expert's, with every token, the last to finish)
  const int blocks = (T + 31) / 32;
  const dim3 grid(blocks < 1024 ? blocks : 1024, groups.n);
  fp8_gather_kernel<<<grid, 256, 0, s>>>(static_cast<const uint8_t*>(x), ldx, groups, offsets, perm, T, k, H,
                                         static_cast<uint8_t*>(dst), stride);
  return cudaGetLastError();
}

bool encode_map_fp8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t row_bytes,
                    uint64_t depth, uint64_t depth_bytes, uint32_t box_rows) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!fn) return false;
  const cuuint32_t dim = depth > 0 ? 3 : 2;
  cuuint64_t dims[3] = {inner, rows, depth};
  cuuint64_t strides[2] = {row_bytes, depth_bytes};
  cuuint32_t box[3] = {(cuuint32_t)kFp8Block, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dim, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ftk

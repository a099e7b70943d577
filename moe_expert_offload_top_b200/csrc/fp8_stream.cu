// Block-scaled fp8 products for few rows: bound by the weights' bytes.
//
// The same functions as fp8_gemm.cu with the operands changed over: 128 weight rows are the
// M of a tcgen05.mma and up to NT token rows its N (16, 32; gate/up 64, product 128), so that one token costs the
// tensor cores N = 16 and not a tile of 128 rows.  TMEM lane = weight row, column = token:
//
//   acc[n][t] += sw[n / 128][kb] sa[t][kb] * (sum over k in block kb of w[n][k] a[t][k])
//
// One CTA per (128 weight rows, expert, NT tokens):
//   warp 0     TMA producer: the weight tile(s) of a block of K (16 KB; gate and up 32 KB) and
//              the tokens' 128 bytes each (gate/up: gathered, a lane asking for four rows),
//              into a ring.  The ring is what reaches the memory's rate: about 200 KB in flight
//              per SM, in one CTA or two.
//   warp 1     MMA issuer, into TMEM buffers in turn (256 columns per CTA).
//   warps 2,3  factors sa * sw of the tokens, four blocks of K at a time, into shared memory.
//   others     sums: a thread owns a weight row; 16 columns at a time leave TMEM and are added
//              with the columns' factors (the same for all lanes: broadcast reads).
// Few tiles (a narrow product) leave SMs without weights to read, so K is split over the CTAs of
// a cluster: each leaves its sums in its shared memory, and rank r adds the columns r * NT / S ..
// of all ranks in rank order (the result does not depend on timing), and stores them.
// Stores: a warp holds 128 consecutive columns of one output row, and so a whole scale block of h.
//
// Every wait is bounded as in fp8_gemm.cu (codes 126-129).  A CTA that gave up stores nothing
// more and leaves out the roles of its later chunks, whose barriers are no longer at the phases
// that `it` and `ch` tell; the cluster barriers are reached by every thread whatever its role met.
#include "fp8.hpp"
#include "fp8_common.cuh"
#include "fp8_mma.cuh"

namespace ftk {
namespace {

constexpr int BK = kFp8Block, WTILE = 128 * BK;
constexpr int FK = 4;             // blocks of K per chunk of factors
constexpr int TMEM_COLS = 256;
constexpr int MAX_STAGES = 8;

template <int COLS>
struct Ctrl {
  uint64_t full[MAX_STAGES], done[MAX_STAGES], tempty[MAX_STAGES], ffull[2], fempty[2], never;
  uint32_t tmem_base;
  int abort;
  alignas(16) float factor[2][FK][COLS];
};

template <int MODE, int NT>
struct Cfg {
  static constexpr int W = MODE == 0 ? 2 : 1;           // weight tiles per block of K
  static constexpr int COLS = W * NT;                   // accumulator columns
  static constexpr int SW = COLS > 32 ? 2 : 1;          // summing warpgroups
  static constexpr int THREADS = 128 + 128 * SW;
  // Two CTAs hide one's set-up and stores behind the other's loads; the gate/up tiles are twice as
  // long and do better with the whole ring to one (FFN of one token, 7 experts: 38.2 -> 35.6 us).
  static constexpr int PER_SM = MODE == 0 || COLS > 32 ? 1 : 2;
  static constexpr int STAGE = W * WTILE + NT * BK;
  // shared memory of an SM (228 KB, 1 KB of it reserved per CTA) over its CTAs
  static constexpr int LIMIT = (228 * 1024) / PER_SM - 1024;
  static constexpr int FIT = (LIMIT - 1024 - (int)sizeof(Ctrl<COLS>)) / STAGE;
  static constexpr int STAGES = FIT < MAX_STAGES ? FIT : MAX_STAGES;
  // Not more buffers than stages: the sums follow the blocks by the phases of the stages'
  // barriers, and may be behind by the number of buffers.
  static constexpr int BUFS = TMEM_COLS / COLS < STAGES ? TMEM_COLS / COLS : STAGES;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + sizeof(Ctrl<COLS>);
  static_assert(STAGES * STAGE >= COLS * 128 * 4, "the sums of a tile wait in the ring's memory");
};

FT_DEVICE void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four consecutive sums, added over the cluster's CTAs in rank order; all loads in flight at once.
FT_DEVICE void total(const float* p, int split, float (&v)[4]) {
  if (split == 1) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    return;
  }
  const uint32_t at = smem_u32(p);
  float f[8][4];
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < split) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(r));
      asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(f[r][0]), "=f"(f[r][1]), "=f"(f[r][2]), "=f"(f[r][3]) : "r"(a) : "memory");
    }
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] = 0.f;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < split) {
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] += f[r][x];
    }
}

template <int MODE, int NT>
__global__ void __launch_bounds__(Cfg<MODE, NT>::THREADS, Cfg<MODE, NT>::PER_SM)
fp8_stream_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ GemmGroups groups,
                  const __grid_constant__ Fp8Gemm p, int split) {
  using C = Cfg<MODE, NT>;
  constexpr int W = C::W, COLS = C::COLS, STAGES = C::STAGES, BUFS = C::BUFS, STAGE = C::STAGE;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Ctrl<COLS>* S = reinterpret_cast<Ctrl<COLS>*>(base + STAGES * STAGE);
  float* part = reinterpret_cast<float*>(base);   // [COLS][128] sums, once the ring is drained
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (p.K + BK - 1) / BK, NB = (p.N + BK - 1) / BK;
  const int rank = split > 1 ? blockIdx.x % split : 0;
  const int n = blockIdx.x / split, g = blockIdx.y;
  const int kb0 = (int)((long long)KB * rank / split), kb1 = (int)((long long)KB * (rank + 1) / split);
  const int e = groups.expert[g], z = groups.z[g];
  int* err = p.err;
  // the same for every CTA of a cluster (they differ in blockIdx.x only)
  const int first = e >= 0 ? p.offsets[e] : p.T * p.k;
  const int rows = e >= 0 ? p.offsets[e + 1] - first : p.T;
  const bool some = (long long)blockIdx.z * NT < rows;

  auto load_weights = [&](int s, int kb) {   // one thread: the stage's barrier and weight tiles
    unsigned char* sw = base + s * STAGE;
    mbar_expect_tx(&S->full[s], STAGE);
    fp8_tma_3d(sw, &maps.b[0], &S->full[s], kb * BK, n * 128, z);
    if (W == 2) fp8_tma_3d(sw + WTILE, &maps.b[1], &S->full[s], kb * BK, n * 128, z);
  };
  // The first weights are on their way before the CTA is set up, and before the kernel that
  // writes the tokens has finished (griddepcontrol below): they depend on neither.
  const int ahead = min(STAGES, kb1 - kb0);
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(&S->full[s], 1);
        mbar_init(&S->done[s], 1);
      }
      for (int b = 0; b < BUFS; ++b) mbar_init(&S->tempty[b], 4 * C::SW);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&S->ffull[b], 2);
        mbar_init(&S->fempty[b], 4 * C::SW);
      }
      mbar_init(&S->never, 1);
      S->abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (some)
        for (int j = 0; j < ahead; ++j) load_weights(j, kb0 + j);
    }
    __syncwarp();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&S->tmem_base)), "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fp8_fence_before();
  __syncthreads();
  fp8_fence_after();
  const uint32_t tmem = S->tmem_base;
  volatile int* abort_flag = &S->abort;
  // gate/up: every CTA is running, so the down product may start to load its weights; down: the
  // rows and scales of h (and what else the launches before it wrote) are complete after the wait.
  if (MODE == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else asm volatile("griddepcontrol.wait;" ::: "memory");

  int it = 0, ch = 0;   // blocks of K and chunks of factors so far
  bool gone = false;    // the CTA gave up in an earlier chunk: the same for all its threads
  for (int t0 = blockIdx.z * NT, chunk = 0; t0 < rows; t0 += gridDim.z * NT, ++chunk) {
    const int valid = min(NT, rows - t0), row0 = first + t0;
    if (gone) {
      // only the barriers
    } else if (warp == 0) {   // -------------------------------------------------- TMA producer
      int tok[4];
      if (MODE == 0) {   // lane l < NT / 4 gathers tokens 4 l .. 4 l + 3; tokens past the last repeat it
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int q = row0 + min(4 * lane + x, valid - 1);
          tok[x] = e < 0 ? q - p.T * p.k : p.perm[q] / p.k;
        }
      }
      int i = it;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int s = i % STAGES;
        if (!warp_wait(&S->done[s], ((i / STAGES) & 1) ^ 1, abort_flag, err, 126)) break;
        unsigned char* sw = base + s * STAGE;
        if (elect_one()) {
          if (i >= ahead) load_weights(s, kb);
          if (MODE == 1) fp8_tma_2d(sw + W * WTILE, &maps.a, &S->full[s], kb * BK, row0);
        }
        __syncwarp();
        if (MODE == 0 && lane < NT / 4)
          fp8_tma_gather4(sw + W * WTILE + lane * 4 * BK, &maps.a, &S->full[s], kb * BK, tok[0], tok[1], tok[2],
                          tok[3]);
        __syncwarp();
      }
      // drain: wait (bounded) until every issued stage has landed
      if (lane == 0)
        for (int j = i - STAGES < it ? it : i - STAGES; j < i; ++j) mbar_drain(&S->full[j % STAGES], (j / STAGES) & 1);
    } else if (warp == 1) {   // -------------------------------------------- MMA issuer
      constexpr uint32_t idesc = fp8_idesc(128, NT);
      const uint64_t desc0 = fp8_desc(smem_u32(base));
      int i = it;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int s = i % STAGES, b = i % BUFS;
        if (!warp_wait2(&S->full[s], (i / STAGES) & 1, &S->tempty[b], ((i / BUFS) & 1) ^ 1, abort_flag, err, 127))
          break;
        fp8_fence_after();
        if (elect_one()) {
          const uint64_t dw = desc0 + (uint32_t)(s * (STAGE >> 4)), da = dw + (W * WTILE >> 4);
#pragma unroll
          for (int w = 0; w < W; ++w)
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              fp8_mma(tmem + b * COLS + w * NT, dw + w * (WTILE >> 4) + 2 * kk, da + 2 * kk, idesc, kk ? 1u : 0u);
          fp8_commit(&S->done[s]);
        }
        __syncwarp();
      }
      // drain: the last commit stands for every MMA issued (the sums may have given up on them)
      if (lane == 0 && i > it) mbar_drain(&S->done[(i - 1) % STAGES], ((i - 1) / STAGES) & 1);
    } else if (warp < 4 && chunk == p.fail_at) {
      never_wait(&S->never, abort_flag, err, 129);
    } else if (warp < 4) {   // --------------------------------------------- factors
      const int t = threadIdx.x - 64;
      constexpr int OWN = (NT + 63) / 64;   // tokens of this thread: t, t + 64
      const float* sa[OWN];
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        int q = row0 + min(t + 64 * i, valid - 1);
        if (MODE == 0) q = e < 0 ? q - p.T * p.k : p.perm[q] / p.k;
        sa[i] = p.a_scales + (long long)q * KB;
      }
      const float* sw[W];
#pragma unroll
      for (int w = 0; w < W; ++w)
        sw[w] = reinterpret_cast<const float*>(p.w_scales[w] + z * p.blob) + (long long)n * KB;
      int c = ch;
      for (int k0 = kb0; k0 < kb1; k0 += FK, ++c) {
        const int b = c & 1;
        float a[OWN][FK], w[W][FK];
#pragma unroll
        for (int j = 0; j < FK; ++j) {
          const int kb = min(k0 + j, kb1 - 1);
#pragma unroll
          for (int i = 0; i < OWN; ++i) a[i][j] = sa[i][kb];
#pragma unroll
          for (int i = 0; i < W; ++i) w[i][j] = sw[i][kb];
        }
        if (!warp_wait(&S->fempty[b], ((c >> 1) & 1) ^ 1, abort_flag, err, 129)) break;
#pragma unroll
        for (int j = 0; j < FK; ++j)
#pragma unroll
          for (int i = 0; i < OWN; ++i)
            if (t + 64 * i < NT) {
#pragma unroll
              for (int x = 0; x < W; ++x) S->factor[b][j][x * NT + t + 64 * i] = a[i][j] * w[x][j];
            }
        warp_arrive(&S->ffull[b]);
      }
    } else {   // ----------------------------------------------------------- sums
      const int q = warp & 3, half = (warp - 4) >> 2;
      const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
      constexpr int C1 = NT / C::SW, CHUNKS = COLS / C::SW / 16;   // columns per weight tile, 16-column chunks
      float acc[CHUNKS * 16];
#pragma unroll
      for (int i = 0; i < CHUNKS * 16; ++i) acc[i] = 0.f;
      auto column = [&](int j) { return (j / (C1 / 16)) * NT + half * C1 + (j % (C1 / 16)) * 16; };
      int i = it, c = ch;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int s = i % STAGES, b = i % BUFS, f = (kb - kb0) % FK, fb = c & 1;
        if (f == 0) ok = warp_wait(&S->ffull[fb], (c >> 1) & 1, abort_flag, err, 128);
        ok = ok && warp_wait(&S->done[s], (i / STAGES) & 1, abort_flag, err, 128);
        if (!ok) break;
        fp8_fence_after();
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
          uint32_t v[16];
          tmem_ld(lane_base + b * COLS + column(j), v);
          tmem_wait(v);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4 x = *reinterpret_cast<const float4*>(&S->factor[fb][f][column(j) + 4 * y]);
            fma_col(acc[16 * j + 4 * y], v[4 * y], x.x);
            fma_col(acc[16 * j + 4 * y + 1], v[4 * y + 1], x.y);
            fma_col(acc[16 * j + 4 * y + 2], v[4 * y + 2], x.z);
            fma_col(acc[16 * j + 4 * y + 3], v[4 * y + 3], x.w);
          }
        }
        fp8_fence_before();
        warp_arrive(&S->tempty[b]);
        if (f == FK - 1 || kb == kb1 - 1) warp_arrive(&S->fempty[fb]);
        c += f == FK - 1 || kb == kb1 - 1;
      }
      // Every block of this CTA has been multiplied: the ring's memory is free for the sums.
      if (ok) {
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
          for (int x = 0; x < 16; ++x) part[(column(j) + x) * 128 + q * 32 + lane] = acc[16 * j + x];
      }
    }
    __syncwarp();
    it += kb1 - kb0;
    ch += (kb1 - kb0 + FK - 1) / FK;
    if (split > 1) cluster_sync(); else __syncthreads();

    // Columns of this rank, added over the ranks: a warp takes a token, a lane four weight rows.
    gone = *abort_flag;   // no role is at work between the barriers
    if (warp >= 4 && !gone) {
      const int c1 = min(NT * (rank + 1) / split, valid);
      const int col = n * 128 + 4 * lane;
#pragma unroll (MODE == 1 ? 2 : 1)
      for (int c = NT * rank / split + warp - 4; c < c1; c += 4 * C::SW) {
        const long long row = row0 + c;
        float v[4];
        total(part + c * 128 + 4 * lane, split, v);
        if constexpr (MODE == 1) {
          const long long at = row * p.ldo + col;
          if (p.out_bf16) {
            uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
            const uint32_t lo = bf16x2(v[0], v[1]), hi = bf16x2(v[2], v[3]);
            if (col + 4 <= p.N && ((uintptr_t)dst & 7) == 0) {
              *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
            } else {
              const uint32_t w[2] = {lo, hi};
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (col + x < p.N) dst[x] = (uint16_t)(w[x >> 1] >> (16 * (x & 1)));
            }
          } else {
            float* dst = static_cast<float*>(p.out) + at;
            if (col + 4 <= p.N && ((uintptr_t)dst & 15) == 0) {
              *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (col + x < p.N) dst[x] = v[x];
            }
          }
        } else {
          float u[4], m = 0.f;
          total(part + (NT + c) * 128 + 4 * lane, split, u);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            v[x] = silu_fast(v[x]) * u[x];
            m = amax_nan(m, v[x]);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = amax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const float sc = fp8_scale(m), inv = 1.0f / sc;
          if (col < p.N)   // N is a multiple of 16
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * p.N + col) =
                e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16;
          if (lane == 0) p.out_scales[row * NB + n] = sc;
        }
      }
    }
    __syncwarp();
    // the sums have been read, by the other ranks too; the ring is the TMA's again
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (split > 1) cluster_sync(); else __syncthreads();
  }
  fp8_fence_before();
  __syncthreads();
  fp8_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

template <int MODE, int NT>
cudaError_t launch_nt(const Fp8Maps& maps, const GemmGroups& groups, const Fp8Gemm& p, int split, int chunks,
                      bool after_gate_up, cudaStream_t s) {
  using C = Cfg<MODE, NT>;
  auto kernel = fp8_stream_kernel<MODE, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.N + 127) / 128 * split), groups.n, chunks);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (after_gate_up) {   // may start while the gate/up kernel finishes (griddepcontrol)
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, maps, groups, p, split);
}

}  // namespace

cudaError_t launch_fp8_stream(int mode, int nt, int split, int chunks, const Fp8Maps& maps, const GemmGroups& groups,
                              const Fp8Gemm& p, bool after_gate_up, cudaStream_t s) {
  if (groups.n <= 0 || p.T <= 0 || p.N <= 0) return cudaSuccess;
  if (mode == 0) {
    switch (nt) {
      case 16: return launch_nt<0, 16>(maps, groups, p, split, chunks, after_gate_up, s);
      case 32: return launch_nt<0, 32>(maps, groups, p, split, chunks, after_gate_up, s);
      default: return launch_nt<0, 64>(maps, groups, p, split, chunks, after_gate_up, s);
    }
  }
  switch (nt) {
    case 16: return launch_nt<1, 16>(maps, groups, p, split, chunks, after_gate_up, s);
    case 32: return launch_nt<1, 32>(maps, groups, p, split, chunks, after_gate_up, s);
    default: return launch_nt<1, 128>(maps, groups, p, split, chunks, after_gate_up, s);
  }
}

}  // namespace ftk

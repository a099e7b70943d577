// Residual addition + root-mean-square norm + e4m3 rows, and the e4m3 rows alone.
//
//   r = round(x + residual)          in x's type: what the residual stream holds
//   y = r / sqrt(mean(r^2) + eps) * w
//   s = max(max |y| / 448, 2^-126)   per 128 columns of a row
//   q = e4m3(y * (1 / s))            round to nearest even
//
// Bound by memory: one pass, each element read once into registers (16 per thread and chunk of
// aligned rows, 8 of others) and written once per output; sums, norm and scales are fp32, and the only roundings to fewer
// bits are the stored r, y and q (q from the fp32 y, not from the stored one).
//
// A row belongs to `tpr` threads (whole warps), so a row's sum is a warp sum plus one exchange
// through shared memory.  Aligned rows: a thread owns 16 consecutive columns per chunk (32-byte
// loads), a scale block is 8 lanes; with 8 columns per thread the two divisions and the
// maximum's exchange, the same work per thread, kept the issue slots half busy.  Others: a warp
// owns two scale blocks per chunk, lane l the columns l, l+32, .. of each, so that element
// loads and byte stores still coalesce.
#include "fp8.hpp"
#include "fp8_common.cuh"

namespace ftk {
namespace {

FT_DEVICE float load1(const void* p, long long i, bool bf16) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
FT_DEVICE void store1(void* p, long long i, float v, bool bf16) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = (uint16_t)bf16x2(v, 0.f);
  else
    static_cast<float*>(p)[i] = v;
}
FT_DEVICE void ld_sector(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p) : "memory");
}
// 16 consecutive elements, 32-byte aligned.
template <bool BF16>
FT_DEVICE void load16(const void* p, long long i, float* v) {
  uint32_t w[8];
  if constexpr (BF16) {
    ld_sector(static_cast<const uint16_t*>(p) + i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) { v[2 * j] = bf16lo(w[j]); v[2 * j + 1] = bf16hi(w[j]); }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ld_sector(static_cast<const float*>(p) + i + 8 * h, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = __uint_as_float(w[j]);
    }
  }
}
template <bool BF16>
FT_DEVICE void store16(void* p, long long i, const float* v) {
  uint32_t w[8];
  if constexpr (BF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = bf16x2(v[2 * j], v[2 * j + 1]);
    st_sector(static_cast<uint16_t*>(p) + i, w);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * h + j]);
      st_sector(static_cast<float*>(p) + i + 8 * h, w);
    }
  }
}
// elements of a thread per chunk; a warp's columns per chunk are 32 times as many
constexpr int elements(bool vec) { return vec ? 16 : 8; }

// blockDim = (tpr, rows per block).  CH: chunks a thread holds.
template <bool BF16, bool NORM, bool VEC, int CH>
__global__ void __launch_bounds__(1024) rows_fp8_kernel(const __grid_constant__ RowsFp8 p) {
  constexpr int E = elements(VEC);
  __shared__ float part[32];
  const int tpr = blockDim.x, t = threadIdx.x;
  const int warp = t >> 5, lane = t & 31, warps = tpr >> 5;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.T;
  const int H = p.H;

  // column of element i of chunk c
  auto col = [&](int c, int i) {
    if constexpr (VEC) return (c * tpr + t) * E + i;
    return ((c * warps + warp) * (E / 4) + (i >> 2)) * kFp8Block + (i & 3) * 32 + lane;
  };
  float v[CH][E];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[c][i] = 0.f;
    if constexpr (VEC) {
      if (live && col(c, 0) < H) {
        load16<BF16>(p.x, row * p.ldx + col(c, 0), v[c]);
        if (NORM && p.residual) {
          float r[E];
          load16<BF16>(p.residual, row * p.ldr + col(c, 0), r);
#pragma unroll
          for (int i = 0; i < E; ++i) v[c][i] += r[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (live && col(c, i) < H) {
          v[c][i] = load1(p.x, row * p.ldx + col(c, i), BF16);
          if (NORM && p.residual) v[c][i] += load1(p.residual, row * p.ldr + col(c, i), BF16);
        }
    }
  }
  if constexpr (NORM) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (p.residual) {
        if constexpr (BF16) {   // the norm is that of the stored stream
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            const uint32_t w = bf16x2(v[c][i], v[c][i + 1]);
            v[c][i] = bf16lo(w);
            v[c][i + 1] = bf16hi(w);
          }
        }
      }
      if (live && p.residual_out) {
        if constexpr (VEC) {
          if (col(c, 0) < H) store16<BF16>(p.residual_out, row * p.ldr + col(c, 0), v[c]);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (col(c, i) < H) store1(p.residual_out, row * p.ldr + col(c, i), v[c][i], BF16);
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i) sum = fmaf(v[c][i], v[c][i], sum);
    }
    sum = warp_sum(sum);
    if (warps > 1) {
      float* mine = part + threadIdx.y * warps;   // rows per block x warps per row <= 32
      if (lane == 0) mine[warp] = sum;
      __syncthreads();
      sum = 0.f;
      for (int w = 0; w < warps; ++w) sum += mine[w];
    }
    const float inv = 1.0f / sqrtf(sum / (float)H + p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (VEC) {
        if (col(c, 0) < H) {
          float w[E];
          load16<BF16>(p.weight, col(c, 0), w);
#pragma unroll
          for (int i = 0; i < E; ++i) v[c][i] = v[c][i] * inv * w[i];
          if (live && p.y) store16<BF16>(p.y, row * H + col(c, 0), v[c]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (col(c, i) < H) {
            v[c][i] = v[c][i] * inv * load1(p.weight, col(c, i), BF16);
            if (live && p.y) store1(p.y, row * H + col(c, i), v[c][i], BF16);
          }
      }
    }
  }
  if (!p.q) return;
  const int blocks = (H + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if constexpr (VEC) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) m = amax_nan(m, v[c][i]);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = amax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float s = fp8_scale(m), inv = 1.0f / s;
      if (live && col(c, 0) < H) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* x = v[c] + 4 * i;
          w[i] = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
        }
        *reinterpret_cast<uint4*>(p.q + row * p.ldq + col(c, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((lane & 7) == 0) p.scales[row * blocks + col(c, 0) / kFp8Block] = s;
      }
    } else {
#pragma unroll
      for (int b = 0; b < E / 4; ++b) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = amax_nan(m, v[c][4 * b + i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = amax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float s = fp8_scale(m), inv = 1.0f / s;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col(c, 4 * b + i) < H)
            p.q[row * p.ldq + col(c, 4 * b + i)] = (uint8_t)e4m3x2(v[c][4 * b + i] * inv, 0.f);
        if (lane == 0 && col(c, 4 * b) < H) p.scales[row * blocks + col(c, 4 * b) / kFp8Block] = s;
      }
    }
  }
}

template <bool BF16, bool NORM, bool VEC>
cudaError_t launch_rows(const RowsFp8& p, int ch, dim3 grid, dim3 block, cudaStream_t s) {
  if (ch == 1)
    rows_fp8_kernel<BF16, NORM, VEC, 1><<<grid, block, 0, s>>>(p);
  else if (VEC || ch == 2)
    rows_fp8_kernel<BF16, NORM, VEC, 2><<<grid, block, 0, s>>>(p);
  else
    rows_fp8_kernel<BF16, NORM, VEC, VEC ? 2 : 4><<<grid, block, 0, s>>>(p);
  return cudaGetLastError();
}
template <bool BF16, bool NORM>
cudaError_t launch_rows(const RowsFp8& p, bool vec, int ch, dim3 grid, dim3 block, cudaStream_t s) {
  return vec ? launch_rows<BF16, NORM, true>(p, ch, grid, block, s)
             : launch_rows<BF16, NORM, false>(p, ch, grid, block, s);
}

}  // namespace

cudaError_t launch_rows_fp8(const RowsFp8& p, bool x_bf16, int num_sms, cudaStream_t s) {
  if (p.T <= 0) return cudaSuccess;
  auto aligned = [](const void* q, int bytes) { return ((uintptr_t)q & (bytes - 1)) == 0; };
  const bool vec = p.H % 16 == 0 && p.ldx % 16 == 0 && aligned(p.x, 32) &&
                   ((!p.residual && !p.residual_out) || p.ldr % 16 == 0) && aligned(p.residual, 32) &&
                   aligned(p.residual_out, 32) && aligned(p.weight, 32) && aligned(p.y, 32) &&
                   (!p.q || (p.ldq % 16 == 0 && aligned(p.q, 16)));
  // One chunk per thread while a block can hold the row's threads: the shortest way from load to
  // store.  Many wide rows with a norm, whose threads wait for one another, take two (8192 x 7168
  // bf16: 110 -> 96 us; without a norm one is better, 30 against 36).
  const int unit = 32 * elements(vec), units = (p.H + unit - 1) / unit;
  const int most = vec && p.weight && p.T > 2 * num_sms ? 8 : 32;
  int ch = 1;
  while (ch < (vec ? 2 : 4) && (units + ch - 1) / ch > most) ch *= 2;
  const int warps = (units + ch - 1) / ch;
  const int rows = warps >= 4 ? 1 : 4 / warps;
  const dim3 block(warps * 32, rows), grid((unsigned)(((long long)p.T + rows - 1) / rows));
  if (p.weight)
    return x_bf16 ? launch_rows<true, true>(p, vec, ch, grid, block, s)
                  : launch_rows<false, true>(p, vec, ch, grid, block, s);
  return x_bf16 ? launch_rows<true, false>(p, vec, ch, grid, block, s)
                : launch_rows<false, false>(p, vec, ch, grid, block, s);
}

}  // namespace ftk

// Residual addition + root-mean-square norm + e4m3 rows, and the e4m3 rows alone.
//
//   r = round(x + residual)          in x's type: what the residual stream holds
//   y = r / sqrt(mean(r^2) + eps) * w
//   s = max(max |y| / 448, 2^-126)   per 128 columns of a row
//   q = e4m3(y * (1 / s))            round to nearest even
//
// Bound by memory: one pass, each element read once into registers (8 per thread and chunk)
// and written once per output; sums, norm and scales are fp32, and the only roundings to fewer
// bits are the stored r, y and q (q from the fp32 y, not from the stored one).
//
// A row belongs to `tpr` threads (whole warps), so a row's sum is a warp sum plus one exchange
// through shared memory.  Aligned rows: a thread owns 8 consecutive columns per chunk (16-byte
// loads), a scale block is 16 lanes.  Others: a warp owns two scale blocks per chunk, lane l
// the columns l, l+32, .. of each, so that element loads and byte stores still coalesce.
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
template <bool BF16>
FT_DEVICE void load8(const void* p, long long i, float* v) {
  if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[2 * j] = bf16lo(w[j]); v[2 * j + 1] = bf16hi(w[j]); }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool BF16>
FT_DEVICE void store8(void* p, long long i, const float* v) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// blockDim = (tpr, rows per block).  CH: chunks of 8 elements a thread holds.
template <bool BF16, bool NORM, bool VEC, int CH>
__global__ void __launch_bounds__(1024) rows_fp8_kernel(const __grid_constant__ RowsFp8 p) {
  __shared__ float part[32];
  const int tpr = blockDim.x, t = threadIdx.x;
  const int warp = t >> 5, lane = t & 31, warps = tpr >> 5;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.T;
  const int H = p.H;

  // column of element i of chunk c
  auto col = [&](int c, int i) {
    if constexpr (VEC) return (c * tpr + t) * 8 + i;
    return ((c * warps + warp) * 2 + (i >> 2)) * kFp8Block + (i & 3) * 32 + lane;
  };
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
    if (!live) continue;
    if constexpr (VEC) {
      if (col(c, 0) < H) load8<BF16>(p.x, row * p.ldx + col(c, 0), v[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col(c, i) < H) v[c][i] = load1(p.x, row * p.ldx + col(c, i), BF16);
    }
  }
  if constexpr (NORM) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (live && p.residual) {
        if constexpr (VEC) {
          if (col(c, 0) < H) {
            float r[8];
            load8<BF16>(p.residual, row * p.ldr + col(c, 0), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] += r[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col(c, i) < H) v[c][i] += load1(p.residual, row * p.ldr + col(c, i), BF16);
        }
        if constexpr (BF16) {   // the norm is that of the stored stream
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint32_t w = bf16x2(v[c][i], v[c][i + 1]);
            v[c][i] = bf16lo(w);
            v[c][i + 1] = bf16hi(w);
          }
        }
      }
      if (live && p.residual_out) {
        if constexpr (VEC) {
          if (col(c, 0) < H) store8<BF16>(p.residual_out, row * p.ldr + col(c, 0), v[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col(c, i) < H) store1(p.residual_out, row * p.ldr + col(c, i), v[c][i], BF16);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[c][i], v[c][i], sum);
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
          float w[8];
          load8<BF16>(p.weight, col(c, 0), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * inv * w[i];
          if (live && p.y) store8<BF16>(p.y, row * H + col(c, 0), v[c]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
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
      for (int i = 0; i < 8; ++i) m = amax_nan(m, v[c][i]);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = amax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float s = fp8_scale(m), inv = 1.0f / s;
      if (live && col(c, 0) < H) {
        uint2 w;
        w.x = e4m3x2(v[c][0] * inv, v[c][1] * inv) | e4m3x2(v[c][2] * inv, v[c][3] * inv) << 16;
        w.y = e4m3x2(v[c][4] * inv, v[c][5] * inv) | e4m3x2(v[c][6] * inv, v[c][7] * inv) << 16;
        *reinterpret_cast<uint2*>(p.q + row * p.ldq + col(c, 0)) = w;
        if ((lane & 15) == 0) p.scales[row * blocks + col(c, 0) / kFp8Block] = s;
      }
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
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
  switch (ch) {
    case 1: rows_fp8_kernel<BF16, NORM, VEC, 1><<<grid, block, 0, s>>>(p); break;
    case 2: rows_fp8_kernel<BF16, NORM, VEC, 2><<<grid, block, 0, s>>>(p); break;
    default: rows_fp8_kernel<BF16, NORM, VEC, 4><<<grid, block, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}
template <bool BF16, bool NORM>
cudaError_t launch_rows(const RowsFp8& p, bool vec, int ch, dim3 grid, dim3 block, cudaStream_t s) {
  return vec ? launch_rows<BF16, NORM, true>(p, ch, grid, block, s)
             : launch_rows<BF16, NORM, false>(p, ch, grid, block, s);
}

}  // namespace

cudaError_t launch_rows_fp8(const RowsFp8& p, bool x_bf16, cudaStream_t s) {
  if (p.T <= 0) return cudaSuccess;
  auto aligned = [](const void* q, int bytes) { return ((uintptr_t)q & (bytes - 1)) == 0; };
  const bool vec = p.H % 8 == 0 && p.ldx % 8 == 0 && aligned(p.x, 16) &&
                   ((!p.residual && !p.residual_out) || p.ldr % 8 == 0) && aligned(p.residual, 16) &&
                   aligned(p.residual_out, 16) && aligned(p.weight, 16) && aligned(p.y, 16) &&
                   (!p.q || (p.ldq % 8 == 0 && aligned(p.q, 8)));
  // units of 256 columns (a warp's chunk); a warp takes ch of them
  const int units = (p.H + 255) / 256;
  // Few rows: one chunk per thread, the shortest chain from load to store.  Many rows: up to
  // four chunks in flight per thread and several rows per SM.
  const int few = p.T <= 2 * 148 ? 32 : 8;
  int ch = 1;
  while (ch < 4 && (units + ch - 1) / ch > few) ch *= 2;
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

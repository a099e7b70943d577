// Internal launch functions of the fp8 operators (host side).
//
// Formats.  Codes are e4m3 bytes.  An activation row carries one fp32 scale per 128
// consecutive columns, a weight matrix one per block of 128 rows x 128 columns; the last
// block of a row or matrix may be partial.  A value is code * scale.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.hpp"

namespace ftk {

constexpr int kFp8Block = 128;
constexpr int kFp8MaxWidth = 32768;   // widest row of the norm and the quantisation
// Largest row, column or pair count of a product: the kernels round such numbers up to tiles, and step
// past the last by less than 2^16, in 32 bits.
constexpr int kFp8MaxCount = 0x7FFFFFFF - 0xFFFF;
inline int fp8_blocks(long long n) { return (int)((n + kFp8Block - 1) / kFp8Block); }

// Rows of x (plus residual) -> norm -> e4m3 rows.  Strides in elements.
struct RowsFp8 {
  const void* x;
  const void* residual;    // may be null
  const void* weight;      // null: no norm
  void* residual_out;      // may be null
  void* y;                 // may be null; contiguous rows
  uint8_t* q;              // may be null
  float* scales;           // [T][blocks of H]
  long long ldx, ldr, ldq; // ldr: rows of residual and residual_out
  int T, H;
  float eps;
};
cudaError_t launch_rows_fp8(const RowsFp8& p, bool x_bf16, int num_sms, cudaStream_t s);

// Tensor maps of one product: A rows (128-byte boxes), and up to two weight matrices
// [slots][rows][K] read 128 K bytes x 128 rows at a time.
struct Fp8Maps {
  CUtensorMap a;
  CUtensorMap b[2];   // gate and up, or the one matrix twice
};

// One grouped product.  Group g's rows and weights as in GemmGroups: routed expert e owns
// rows offsets[e] .. offsets[e+1], expert -1 the rows T*k .. T*k+T-1 (a dense product is
// that group alone with k = 0).
struct Fp8Gemm {
  const float* a_scales;      // [rows][KB]; gate/up: [T][KB], the token's row
  const uint8_t* w_scales[2]; // scales of slot 0's matrices; slot z is blob bytes further
  long long blob;
  const int* offsets;
  const int* perm;            // gate/up: token of pair row q = perm[q] / k
  int T, k, N, K;             // N: output columns (gate/up: I)
  void* out;                  // gate/up: codes [rows][N]; else f32 or bf16 rows of ldo elements
  float* out_scales;          // gate/up: [rows][NB]
  long long ldo;
  int out_bf16;
  int* err;
  int fail_at = -1;           // tests: the chunk or tile of a CTA in which a role waits for what never comes
};
// mode 0: gate/up + SwiGLU + quantisation, mode 1: the product itself.
cudaError_t launch_fp8_gemm(int mode, const Fp8Maps& maps, const GemmGroups& groups, const Fp8Gemm& p, int num_sms,
                            cudaStream_t s);
// The same product with the weights as the tensor cores' M, for few rows (fp8_stream.cu): nt
// tokens (16, 32; mode 0: 64, mode 1: 128) per CTA, K split over clusters of `split` CTAs (1 .. 8, at most
// the blocks of K), `chunks` CTAs sharing a group's token chunks.  maps.a: mode 0 boxes of one
// row of x, mode 1 of nt rows.  after_gate_up: this launch may start, and load weights, while the launch
// before it on the stream finishes, and waits for that one's end before it reads its rows.  The
// launch before it must itself start behind the end of every launch that writes those rows or
// offsets (no programmatic start of its own), as all gate/up launches do.
cudaError_t launch_fp8_stream(int mode, int nt, int split, int chunks, const Fp8Maps& maps, const GemmGroups& groups,
                              const Fp8Gemm& p, bool after_gate_up, cudaStream_t s);
// dst + q * stride = the H bytes of pair q's token row, for the pairs of the groups.
cudaError_t launch_fp8_gather(const void* x, long long ldx, const GemmGroups& groups, const int* offsets,
                              const int* perm, int T, int k, int H, void* dst, long long stride, cudaStream_t s);
// uint8 tensor map [depth][rows][inner], 128-byte swizzle, boxes of 128 bytes x box_rows x 1.
bool encode_map_fp8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t row_bytes,
                    uint64_t depth, uint64_t depth_bytes, uint32_t box_rows);

}  // namespace ftk

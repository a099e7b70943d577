// C entry points of the fp8 operators (include/ftmoe.h): argument checks, tensor maps, launches.
#include <string>

#include "fp8.hpp"
#include "ftmoe.h"

namespace ftk {
void set_step_error(const std::string& msg);   // message behind ft_last_error(NULL)
}

namespace {

int bad(const char* call, const char* why) {
  ftk::set_step_error(std::string(call) + ": " + why);
  return FT_ERR_INVALID;
}
int failed(const char* call, const char* what, cudaError_t e) {
  ftk::set_step_error(std::string(call) + ": " + what + cudaGetErrorString(e));
  return FT_ERR_CUDA;
}
bool aligned(const void* p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// The output must be memory of the current device: the launch would run there, and a host
// address or another GPU's memory would fault it.
int check_device(const char* call, const void* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  cudaPointerAttributes at{};
  if (e == cudaSuccess) e = cudaPointerGetAttributes(&at, out);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return failed(call, "no device: ", e);
  }
  if ((at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) ||
      (at.type == cudaMemoryTypeDevice && at.device != dev))
    return bad(call, "the output is not memory of the current device");
  return FT_OK;
}
int num_sms() {
  int dev = 0, n = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// How a product of `rows` rows per group runs: nt > 0 on the streaming kernel with nt tokens per
// CTA, nt = 0 on the tiles of 128 rows.
struct Plan {
  int nt, split, chunks;
};
Plan plan(int mode, long long rows, int groups, int N, int K, int sms) {
  Plan pl{0, 1, 1};
  if (rows > (mode == 0 ? 64 : 256)) return pl;
  const int most = mode == 0 ? 64 : 128;
  pl.nt = 16;
  while (pl.nt < rows && pl.nt < most) pl.nt *= 2;
  pl.chunks = (int)((rows + pl.nt - 1) / pl.nt);
  const long long tiles = (long long)ftk::fp8_blocks(N) * groups * pl.chunks;
  const int kb = ftk::fp8_blocks(K);
  while (pl.split < 8 && 3 * tiles * pl.split < 2 * sms && kb >= 4 * pl.split) pl.split *= 2;
  return pl;
}

int rows_call(const char* call, const ftk::RowsFp8& p, int x_is_bf16, void* stream) {
  const uintptr_t es = x_is_bf16 ? 2 : 4;
  if (p.T < 0 || p.H < 1) return bad(call, "invalid size");
  if (p.H > ftk::kFp8MaxWidth) return bad(call, "H is above 32768");
  if (p.ldx < p.H || (p.q && p.ldq < p.H) || ((p.residual || p.residual_out) && p.ldr < p.H))
    return bad(call, "a row stride is smaller than H");
  if (p.T == 0) return FT_OK;
  if (!p.x || (!p.q && !p.y) || (p.q && !p.scales)) return bad(call, "null pointer");
  if (!aligned(p.x, es) || !aligned(p.residual, es) || !aligned(p.weight, es) || !aligned(p.residual_out, es) ||
      !aligned(p.y, es) || !aligned(p.scales, 4))
    return bad(call, "a buffer is not aligned to its elements");
  const int rc = check_device(call, p.q ? static_cast<const void*>(p.q) : p.y);
  if (rc != FT_OK) return rc;
  const cudaError_t e = ftk::launch_rows_fp8(p, x_is_bf16 != 0, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FT_OK : failed(call, "launch: ", e);
}

}  // namespace

extern "C" {

int ft_rmsnorm_fp8(const void* x, long long ldx, const void* residual, long long ldr, const void* weight,
                   int x_is_bf16, int T, int H, float eps, void* residual_out, void* y, void* q, long long ldq,
                   float* scales, void* stream) {
  const char* call = "ft_rmsnorm_fp8";
  if (!(eps >= 0.0f)) return bad(call, "eps must be a number of at least 0");
  if (T > 0 && !weight) return bad(call, "null pointer");
  const ftk::RowsFp8 p{x, residual, weight, residual_out, y, static_cast<uint8_t*>(q), scales, ldx, ldr, ldq, T, H, eps};
  return rows_call(call, p, x_is_bf16, stream);
}

int ft_quantize_fp8(const void* x, long long ldx, int x_is_bf16, int T, int H, void* q, long long ldq, float* scales,
                    void* stream) {
  if (T > 0 && !q) return bad("ft_quantize_fp8", "null pointer");
  const ftk::RowsFp8 p{x, nullptr, nullptr, nullptr, nullptr, static_cast<uint8_t*>(q), scales, ldx, 0, ldq, T, H, 0.f};
  return rows_call("ft_quantize_fp8", p, x_is_bf16, stream);
}

int ft_gemm_fp8(const void* a, long long lda, const float* a_scales, const void* w, long long ldw,
                const float* w_scales, int M, int N, int K, int out_is_bf16, void* out, long long ldo, int* err,
                void* stream) {
  const char* call = "ft_gemm_fp8";
  if (M < 0 || N < 0 || K < 1) return bad(call, "invalid size");
  if (lda < K || ldw < K || ldo < N) return bad(call, "a row stride is smaller than the row");
  if (lda % 16 || ldw % 16) return bad(call, "lda and ldw must be multiples of 16");
  if (M == 0 || N == 0) return FT_OK;
  if (!a || !a_scales || !w || !w_scales || !out || !err) return bad(call, "null pointer");
  if (!aligned(a, 16) || !aligned(w, 16)) return bad(call, "a and w must be 16-byte aligned");
  if (!aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(out, out_is_bf16 ? 2 : 4) || !aligned(err, 4))
    return bad(call, "a buffer is not aligned to its elements");
  const int rc = check_device(call, out);
  if (rc != FT_OK) return rc;
  const int sms = num_sms();
  const Plan pl = plan(1, M, 1, N, K, sms);
  ftk::Fp8Maps m;
  if (!ftk::encode_map_fp8(&m.a, a, K, M, lda, 0, 0, pl.nt ? pl.nt : 128) ||
      !ftk::encode_map_fp8(&m.b[0], w, K, N, ldw, 1, (uint64_t)ldw * N, 128)) {
    ftk::set_step_error(std::string(call) + ": cuTensorMapEncodeTiled failed");
    return FT_ERR_CUDA;
  }
  m.b[1] = m.b[0];
  ftk::GemmGroups groups;
  groups.n = 1;
  groups.expert[0] = -1;   // all M rows
  groups.z[0] = 0;
  const uint8_t* ws = reinterpret_cast<const uint8_t*>(w_scales);
  const ftk::Fp8Gemm p{a_scales, {ws, ws}, 0, nullptr, nullptr, M, 0, N, K, out, nullptr, ldo, out_is_bf16 != 0, err};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pl.nt ? ftk::launch_fp8_stream(1, pl.nt, pl.split, pl.chunks, m, groups, p, false, s)
                              : ftk::launch_fp8_gemm(1, m, groups, p, sms, s);
  return e == cudaSuccess ? FT_OK : failed(call, "launch: ", e);
}

size_t ft_fp8_blob_bytes(int H, int I) {
  if (H < 16 || I < 16 || H % 16 || I % 16) return 0;
  const size_t scales = (size_t)ftk::fp8_blocks(H) * ftk::fp8_blocks(I);
  return (3 * ((size_t)H * I + 4 * scales) + 15) / 16 * 16;
}

int ft_expert_ffn_fp8(const void* x, long long ldx, const float* x_scales, int T, int H, int I, int top_k,
                      const void* weights, int n_slots, const int* experts, const int* slots, int n_list,
                      const int* offsets, const int* perm, void* h, float* h_scales, float* y, int* err,
                      void* stream) {
  const char* call = "ft_expert_ffn_fp8";
  if (T < 0 || top_k < 1 || top_k > FT_MAX_TOPK || n_list < 0 || n_list > ftk::kMaxList || n_slots < 1)
    return bad(call, "invalid size");
  if (H < 16 || I < 16 || H % 16 || I % 16) return bad(call, "H and I must be multiples of 16");
  if ((long long)T * (top_k + 1) > 0x7FFFFFFF) return bad(call, "T * (top_k + 1) is above 2^31 - 1");
  if (ldx < H || ldx % 16) return bad(call, "ldx must be a multiple of 16 of at least H");
  if (T == 0 || n_list == 0) return FT_OK;
  if (!x || !x_scales || !weights || !experts || !slots || !offsets || !perm || !h || !h_scales || !y || !err)
    return bad(call, "null pointer");
  if (!aligned(x, 16) || !aligned(weights, 16) || !aligned(h, 16) || !aligned(y, 16))
    return bad(call, "x, weights, h and y must be 16-byte aligned");
  if (!aligned(x_scales, 4) || !aligned(h_scales, 4) || !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(err, 4))
    return bad(call, "a buffer is not aligned to its elements");
  ftk::GemmGroups groups;
  groups.n = n_list;
  bool seen[FT_MAX_EXPERTS + 1] = {};
  for (int i = 0; i < n_list; ++i) {
    if (experts[i] < -1 || experts[i] >= FT_MAX_EXPERTS || slots[i] < 0 || slots[i] >= n_slots)
      return bad(call, "bad expert list entry");
    if (seen[experts[i] + 1]) return bad(call, "an expert is listed twice");   // its rows would be written twice
    seen[experts[i] + 1] = true;
    groups.expert[i] = experts[i];
    groups.z[i] = slots[i];
  }
  const int rc = check_device(call, y);
  if (rc != FT_OK) return rc;
  const uint64_t rows = (uint64_t)T * top_k + T, n = (uint64_t)H * I, blob = ft_fp8_blob_bytes(H, I);
  const size_t sb = 4 * (size_t)ftk::fp8_blocks(H) * ftk::fp8_blocks(I);
  const uint8_t* w = static_cast<const uint8_t*>(weights);
  // pairs per listed expert, were they spread evenly
  const int sms = num_sms();
  const long long each = ((long long)T * top_k + n_list - 1) / n_list;
  const Plan pu = plan(0, each, n_list, I, H, sms), pd = plan(1, each > 64 ? 257 : each, n_list, H, I, sms);
  ftk::Fp8Maps up, down;
  if (!(pu.nt ? ftk::encode_map_fp8(&up.a, x, H, T, ldx, 0, 0, 1)
              : ftk::encode_map_fp8(&up.a, y, H, rows, 4ull * H, 0, 0, 128)) ||
      !ftk::encode_map_fp8(&up.b[0], w, H, I, H, n_slots, blob, 128) ||
      !ftk::encode_map_fp8(&up.b[1], w + n, H, I, H, n_slots, blob, 128) ||
      !ftk::encode_map_fp8(&down.a, h, I, rows, I, 0, 0, pd.nt ? pd.nt : 128) ||
      !ftk::encode_map_fp8(&down.b[0], w + 2 * n, I, H, I, n_slots, blob, 128)) {
    ftk::set_step_error(std::string(call) + ": cuTensorMapEncodeTiled failed");
    return FT_ERR_CUDA;
  }
  down.b[1] = down.b[0];
  const uint8_t* ws = w + 3 * n;
  const ftk::Fp8Gemm g{x_scales, {ws, ws + sb}, (long long)blob, offsets, perm, T, top_k, I, H, h, h_scales, I, 0, err};
  const ftk::Fp8Gemm d{h_scales, {ws + 2 * sb, ws + 2 * sb}, (long long)blob, offsets, perm, T, top_k, H, I,
                       y, nullptr, H, 0, err};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (pu.nt) {
    e = ftk::launch_fp8_stream(0, pu.nt, pu.split, pu.chunks, up, groups, g, false, s);
  } else {
    // the pairs' token rows wait in the rows of y that the down product writes last
    e = ftk::launch_fp8_gather(x, ldx, groups, offsets, perm, T, top_k, H, y, 4ll * H, sms, s);
    if (e == cudaSuccess) e = ftk::launch_fp8_gemm(0, up, groups, g, sms, s);
  }
  if (e == cudaSuccess)
    e = pd.nt ? ftk::launch_fp8_stream(1, pd.nt, pd.split, pd.chunks, down, groups, d, pu.nt > 0, s)
              : ftk::launch_fp8_gemm(1, down, groups, d, sms, s);
  return e == cudaSuccess ? FT_OK : failed(call, "launch: ", e);
}

}  // extern "C"

// C entry points of the fp8 operators (include/ftmoe.h): argument checks, tensor maps, launches.
#include <algorithm>
#include <atomic>
#include <cmath>
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

// The output must be memory of the current device, which is returned in dev: the launch would run
// there, and a host address or another GPU's memory would fault it.
int check_device(const char* call, const void* out, int& dev) {
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
// SMs of a device; asked for once, as they do not change.
int num_sms(int dev) {
  static std::atomic<int> known[64];
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// How a product of `rows` rows per group runs: nt > 0 on the streaming kernel with nt tokens per
// CTA, nt = 0 on the tiles of 128 rows.
struct Plan {
  int nt, split, chunks;
};
// The plan of the least estimated time, in us as measured on a B200.  A CTA of the streaming kernel
// takes a time of its own (more where K is split: the exchange of the sums) and a time per block of
// K, less of it where two share an SM (`pair`); an SM runs its CTAs in turn.  The tiles take a
// fixed time, and per wave a time per block and one for the stores.  No plan is faster than the
// weights' bytes.  It knows the average of a routing only: where one expert has most tokens, its
// CTAs take them in turn while the others have left.  What it decides, measured (us, bf16 out):
//   4096 x 4096 weights, 1 row: 16 tokens per CTA, K in four 6.7; tiles 18.0
//   200 rows: 128 tokens, K in two 16.4; tiles 20.6.  384 rows: tiles 20.8; 128 tokens 22.4
//   100 x 512 x 512: 16 tokens, K whole 4.7; K in four 4.5, 128 tokens 6.9, tiles 7.5
//   gate/up with 64 tokens, FFN of 4096 x 128 x 128 one expert: 19.3; tiles 24.5 (4096 x 4096 x 128: 54 and 62)
Plan plan(int mode, long long rows, int groups, int N, int K, int sms, bool aligned_rows) {
  struct Kind {
    int nt;
    double own, own_split, alone, pair;
  };
  static const Kind product[3] = {{16, 1.0, 2.0, 0.25, 0.175}, {32, 1.2, 2.0, 0.33, 0.25}, {128, 3.4, 5.2, 0.54, 0.54}};
  static const Kind gate_up[3] = {{16, 1.0, 2.0, 0.40, 0.30}, {32, 1.2, 2.0, 0.53, 0.40}, {64, 3.4, 5.2, 0.80, 0.80}};
  const int kb = ftk::fp8_blocks(K), tn = mode == 0 ? 128 : 256;
  const long long tiles = (rows + 127) / 128 * ((N + tn - 1) / tn) * groups;
  const double bytes = 2.2 + (mode == 0 ? 2.0 : 1.0) * N * K * groups / 6.0e6;
  // the tiles of gate/up: after a launch that copies the rows, and no early start for the down product
  const double fixed = mode == 0 ? 10.0 : 5.0;
  Plan best{0, 1, 1};
  double least = fixed + (double)((tiles + sms - 1) / sms) * (0.45 * kb + (aligned_rows ? 1.5 : 8.0));
  if (least < bytes + fixed - 2.2) least = bytes + fixed - 2.2;
  for (const Kind& k : mode == 0 ? gate_up : product) {
    const long long chunks = (rows + k.nt - 1) / k.nt;
    if (chunks > 64) continue;
    for (int split = 1; split <= 8 && split <= kb; split *= 2) {
      const long long ctas = ftk::fp8_blocks(N) * groups * chunks * split, turns = (ctas + sms - 1) / sms;
      const double per_block = turns == 1 ? k.alone : k.pair;
      double t = 2.2 + turns * ((split == 1 ? k.own : k.own_split) + per_block * ((kb + split - 1) / split));
      if (t < bytes) t = bytes;
      if (t < least) {
        least = t;
        best = Plan{k.nt, split, (int)chunks};
      }
    }
  }
  return best;
}
// The chunk or tile of every CTA that a test lets fail; -1: none.
bool valid_fail(int fail_at) { return fail_at >= -1 && fail_at <= (1 << 20); }
// A plan that the kernels can run: the token counts of `mode`, K in 1, 2, 4 or 8 parts of a block at least.
bool valid(int mode, const Plan& p, int K) {
  if (p.nt == 0) return true;
  if (p.nt != 16 && p.nt != 32 && p.nt != (mode == 0 ? 64 : 128)) return false;
  if (p.split < 1 || p.split > 8 || (p.split & (p.split - 1)) || p.split > ftk::fp8_blocks(K)) return false;
  return p.chunks >= 1 && p.chunks <= 64;
}

int rows_call(const char* call, const ftk::RowsFp8& p, int x_is_bf16, void* stream) {
  const uintptr_t es = x_is_bf16 ? 2 : 4;
  if (p.T < 0 || p.H < 1) return bad(call, "invalid size");
  if (p.H > ftk::kFp8MaxWidth) return bad(call, "H is above 32768");
  if (p.ldx < p.H || (p.q && p.ldq < p.H) || ((p.residual || p.residual_out) && p.ldr < p.H))
    return bad(call, "a row stride is smaller than H");
  if (p.T > 1 && p.residual_out && p.residual_out == p.x && p.ldx != p.ldr)   // rows written before they are read
    return bad(call, "residual_out may be x only where ldx and ldr are the same stride");
  if (p.T == 0) return FT_OK;
  if (!p.x || (!p.q && !p.y) || (p.q && !p.scales)) return bad(call, "null pointer");
  if (!aligned(p.x, es) || !aligned(p.residual, es) || !aligned(p.weight, es) || !aligned(p.residual_out, es) ||
      !aligned(p.y, es) || !aligned(p.scales, 4))
    return bad(call, "a buffer is not aligned to its elements");
  int dev = 0;
  const int rc = check_device(call, p.q ? static_cast<const void*>(p.q) : p.y, dev);
  if (rc != FT_OK) return rc;
  const cudaError_t e = ftk::launch_rows_fp8(p, x_is_bf16 != 0, num_sms(dev), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FT_OK : failed(call, "launch: ", e);
}

// ft_gemm_fp8, by `forced` where that is given.
int gemm_fp8(const char* call, const void* a, long long lda, const float* a_scales, const void* w, long long ldw,
             const float* w_scales, int M, int N, int K, int out_is_bf16, void* out, long long ldo, int* err,
             const Plan* forced, int fail_at, void* stream) {
  if (M < 0 || N < 0 || K < 1) return bad(call, "invalid size");
  if (M > ftk::kFp8MaxCount || N > ftk::kFp8MaxCount || K > ftk::kFp8MaxCount)
    return bad(call, "M, N or K is above 2^31 - 2^16");
  if (lda < K || ldw < K || ldo < N) return bad(call, "a row stride is smaller than the row");
  if (lda % 16 || ldw % 16) return bad(call, "lda and ldw must be multiples of 16");
  if (forced && (!valid(1, *forced, K) || !valid_fail(fail_at))) return bad(call, "no such plan");
  if (M == 0 || N == 0) return FT_OK;
  if (!a || !a_scales || !w || !w_scales || !out || !err) return bad(call, "null pointer");
  if (!aligned(a, 16) || !aligned(w, 16)) return bad(call, "a and w must be 16-byte aligned");
  if (!aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(out, out_is_bf16 ? 2 : 4) || !aligned(err, 4))
    return bad(call, "a buffer is not aligned to its elements");
  int dev = 0;
  const int rc = check_device(call, out, dev);
  if (rc != FT_OK) return rc;
  const int sms = num_sms(dev);
  const Plan pl =
      forced ? *forced : plan(1, M, 1, N, K, sms, ldo * (out_is_bf16 ? 2 : 4) % 16 == 0 && aligned(out, 16));
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
  const ftk::Fp8Gemm p{a_scales, {ws, ws}, 0, nullptr, nullptr, M, 0, N, K, out, nullptr, ldo, out_is_bf16 != 0, err,
                       fail_at};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = pl.nt ? ftk::launch_fp8_stream(1, pl.nt, pl.split, pl.chunks, m, groups, p, false, s)
                              : ftk::launch_fp8_gemm(1, m, groups, p, sms, s);
  return e == cudaSuccess ? FT_OK : failed(call, "launch: ", e);
}

// ft_expert_ffn_fp8; by forced[0] (gate/up) and forced[1] (down) where that is given.
int expert_ffn_fp8(const char* call, const void* x, long long ldx, const float* x_scales, int T, int H, int I,
                   int top_k, const void* weights, int n_slots, const int* experts, const int* slots, int n_list,
                   const int* offsets, const int* perm, void* h, float* h_scales, float* y, int* err,
                   const Plan* forced, int fail_at, void* stream) {
  if (T < 0 || top_k < 1 || top_k > FT_MAX_TOPK || n_list < 0 || n_list > ftk::kMaxList || n_slots < 1)
    return bad(call, "invalid size");
  if (H < 16 || I < 16 || H % 16 || I % 16) return bad(call, "H and I must be multiples of 16");
  if (H > ftk::kFp8MaxCount || I > ftk::kFp8MaxCount) return bad(call, "H or I is above 2^31 - 2^16");
  if ((long long)T * (top_k + 1) > ftk::kFp8MaxCount) return bad(call, "T * (top_k + 1) is above 2^31 - 2^16");
  if (ldx < H || ldx % 16) return bad(call, "ldx must be a multiple of 16 of at least H");
  if (forced && (!valid(0, forced[0], H) || !valid(1, forced[1], I) || !valid_fail(fail_at)))
    return bad(call, "no such plan");
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
  int dev = 0;
  const int rc = check_device(call, y, dev);
  if (rc != FT_OK) return rc;
  const uint64_t pairs = (uint64_t)T * top_k + T, n = (uint64_t)H * I, blob = ft_fp8_blob_bytes(H, I);
  const size_t sb = 4 * (size_t)ftk::fp8_blocks(H) * ftk::fp8_blocks(I);
  const uint8_t* w = static_cast<const uint8_t*>(weights);
  const int sms = num_sms(dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint8_t* ws = w + 3 * n;
  const ftk::Fp8Gemm g{x_scales, {ws, ws + sb}, (long long)blob, offsets, perm, T, top_k, I, H, h, h_scales, I, 0, err,
                       fail_at};
  const ftk::Fp8Gemm d{h_scales, {ws + 2 * sb, ws + 2 * sb}, (long long)blob, offsets, perm, T, top_k, H, I,
                       y, nullptr, H, 0, err, fail_at};
  // The launches of one product of some of the groups, `rows` rows each.  The gate/up tiles find
  // the pairs' token rows in the rows of y that the down product writes last.
  const char* what = "launch: ";
  auto product = [&](int mode, const ftk::GemmGroups& gr, long long rows, bool early) -> cudaError_t {
    const Plan pl = forced ? forced[mode] : plan(mode, rows, gr.n, mode == 0 ? I : H, mode == 0 ? H : I, sms, true);
    const uint32_t box = pl.nt ? pl.nt : 128;
    ftk::Fp8Maps m;
    bool ok;
    if (mode == 0) {
      ok = (pl.nt ? ftk::encode_map_fp8(&m.a, x, H, T, ldx, 0, 0, 1)
                  : ftk::encode_map_fp8(&m.a, y, H, pairs, 4ull * H, 0, 0, box)) &&
           ftk::encode_map_fp8(&m.b[0], w, H, I, H, n_slots, blob, 128) &&
           ftk::encode_map_fp8(&m.b[1], w + n, H, I, H, n_slots, blob, 128);
    } else {
      ok = ftk::encode_map_fp8(&m.a, h, I, pairs, I, 0, 0, box) &&
           ftk::encode_map_fp8(&m.b[0], w + 2 * n, I, H, I, n_slots, blob, 128);
      m.b[1] = m.b[0];
    }
    if (!ok) {
      what = "cuTensorMapEncodeTiled: ";
      return cudaErrorInvalidValue;
    }
    if (pl.nt) return ftk::launch_fp8_stream(mode, pl.nt, pl.split, pl.chunks, m, gr, mode == 0 ? g : d, early, s);
    cudaError_t e = cudaSuccess;
    if (mode == 0) e = ftk::launch_fp8_gather(x, ldx, gr, offsets, perm, T, top_k, H, y, 4ll * H, s);
    return e == cudaSuccess ? ftk::launch_fp8_gemm(mode, m, gr, mode == 0 ? g : d, sms, s) : e;
  };
  // Pairs of a routed expert: the even share and three times its square root, the spread of a
  // random routing (an expert with more takes its CTAs longer).  The shared expert has T.
  const int routed = n_list - (seen[0] ? 1 : 0);
  const double even = routed ? (double)T * top_k / routed : 0.0;
  const long long each = std::min((long long)T, (long long)std::ceil(even + 3.0 * std::sqrt(even)));
  cudaError_t e;
  if (!forced && seen[0] && routed && T > 16 && T > 2 * each && plan(0, each, routed, I, H, sms, true).nt) {
    // far more rows in the shared expert, and the others stream: its products are launched by
    // themselves (100 tokens, 64 experts, top 4: 342 -> 279 us); the tiles take any mix at once
    ftk::GemmGroups some, shared;
    some.n = 0;
    shared.n = 1;
    for (int i = 0; i < n_list; ++i) {
      ftk::GemmGroups& to = experts[i] < 0 ? shared : some;
      const int at = experts[i] < 0 ? 0 : some.n++;
      to.expert[at] = groups.expert[i];
      to.z[at] = groups.z[i];
    }
    e = product(0, some, each, false);
    if (e == cudaSuccess) e = product(0, shared, T, false);
    if (e == cudaSuccess) e = product(1, some, each, true);
    if (e == cudaSuccess) e = product(1, shared, T, false);
  } else {
    const long long rows = std::max(each, seen[0] ? (long long)T : 0ll);
    e = product(0, groups, rows, false);
    if (e == cudaSuccess) e = product(1, groups, rows, true);
  }
  return e == cudaSuccess ? FT_OK : failed(call, what, e);
}

}  // namespace

extern "C" {

int ft_rmsnorm_fp8(const void* x, long long ldx, const void* residual, long long ldr, const void* weight,
                   int x_is_bf16, int T, int H, float eps, void* residual_out, void* y, void* q, long long ldq,
                   float* scales, void* stream) {
  const char* call = "ft_rmsnorm_fp8";
  if (!(eps >= 0.0f)) return bad(call, "eps must be a number of at least 0");
  if (T > 0 && !weight) return bad(call, "null pointer");
  const ftk::RowsFp8 p{x,   residual, weight, residual_out, y, static_cast<uint8_t*>(q), scales,
                       ldx, ldr,      ldq,    T,            H, eps};
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
  return gemm_fp8("ft_gemm_fp8", a, lda, a_scales, w, ldw, w_scales, M, N, K, out_is_bf16, out, ldo, err, nullptr,
                  -1, stream);
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
  return expert_ffn_fp8("ft_expert_ffn_fp8", x, ldx, x_scales, T, H, I, top_k, weights, n_slots, experts, slots, n_list,
                        offsets, perm, h, h_scales, y, err, nullptr, -1, stream);
}

int ft_debug_fp8_plan(int mode, int rows, int groups, int N, int K, int num_sms, int rows_aligned, int* plan3) {
  if ((mode != 0 && mode != 1) || rows < 0 || groups < 1 || N < 1 || K < 1 || num_sms < 1 || !plan3 ||
      rows > ftk::kFp8MaxCount || N > ftk::kFp8MaxCount || K > ftk::kFp8MaxCount)
    return bad("ft_debug_fp8_plan", "invalid argument");
  const Plan p = plan(mode, rows, groups, N, K, num_sms, rows_aligned != 0);
  plan3[0] = p.nt;
  plan3[1] = p.split;
  plan3[2] = p.chunks;
  return FT_OK;
}

int ft_debug_gemm_fp8(const void* a, long long lda, const float* a_scales, const void* w, long long ldw,
                      const float* w_scales, int M, int N, int K, int out_is_bf16, void* out, long long ldo, int* err,
                      const int* plan3, int fail_at, void* stream) {
  if (!plan3) return bad("ft_debug_gemm_fp8", "null pointer");
  const Plan p{plan3[0], plan3[1], plan3[2]};
  return gemm_fp8("ft_debug_gemm_fp8", a, lda, a_scales, w, ldw, w_scales, M, N, K, out_is_bf16, out, ldo, err, &p,
                  fail_at, stream);
}

int ft_debug_expert_ffn_fp8(const void* x, long long ldx, const float* x_scales, int T, int H, int I, int top_k,
                            const void* weights, int n_slots, const int* experts, const int* slots, int n_list,
                            const int* offsets, const int* perm, void* h, float* h_scales, float* y, int* err,
                            const int* plan6, int fail_at, void* stream) {
  if (!plan6) return bad("ft_debug_expert_ffn_fp8", "null pointer");
  const Plan p[2] = {{plan6[0], plan6[1], plan6[2]}, {plan6[3], plan6[4], plan6[5]}};
  return expert_ffn_fp8("ft_debug_expert_ffn_fp8", x, ldx, x_scales, T, H, I, top_k, weights, n_slots, experts, slots,
                        n_list, offsets, perm, h, h_scales, y, err, p, fail_at, stream);
}

}  // extern "C"

// C ABI of the gated feed-forward block (tpmlp_gated_forward, tpmlp_gated_backward): the checks of the arguments and the
// sequence of products. The products with an elementwise part are in gemm_tc.cu (kEpiGate, kEpiGateGrad).
// Y and D go from one product to the next in bf16, as Y and D of the GeLU MLP do: the tensor core's operands, and half the bytes. That
// takes the results from 0.0017 of their norm off 64 bits (the rounding of the result alone) to 0.0023: two independent roundings of
// 2^-8 / sqrt(3) of a value at most, some 0.0017 each over a matrix, and sqrt(2) of that. Everything between is fp32.
#include <cuda_runtime.h>

#include "abi_checks.h"

namespace tpmlp {
namespace {

tpmlp_status check_gated_shape(int64_t n, int64_t d, int64_t m, int t, int act, tpmlp_dtype dt) {
  if (dt != TPMLP_BF16) return err(TPMLP_ERR_DTYPE, "the gated block runs on the bf16 tensor-core path only");
  if (act != TPMLP_GATE_GELU_ERF && act != TPMLP_GATE_GELU_TANH && act != TPMLP_GATE_SILU)
    return err(TPMLP_ERR_INVALID, "unknown gate activation");
  if (n < 0 || d < 1 || m < 1) return err(TPMLP_ERR_SHAPE, "need n >= 0, d >= 1, m >= 1");
  if (t < 1) return err(TPMLP_ERR_SHAPE, "t must be >= 1");
  if (m % t != 0) return err(TPMLP_ERR_SHAPE, "m is not divisible by t (shards are an equal split)");
  if (d % 8 != 0 || (m / t) % 8 != 0) return err(TPMLP_ERR_SHAPE, "d and m / t must be multiples of 8");
  if (n > INT32_MAX - 1024 || d > INT32_MAX - 1024 || m > (1 << 30) - 1024)
    return err(TPMLP_ERR_SHAPE, "n and d must be below 2^31 - 1024, m below 2^30 - 1024");
  return TPMLP_OK;
}

Region matrix(const void* p, int64_t rows, int64_t cols, int64_t size = 2) {
  return flat_region(p, rows * cols, size);  // both below 2^31
}

// The products behind a call's first one: each is launched as a programmatic dependent of the kernel in front of it, and
// waits for that kernel's end before it touches memory.
EpiParams plain(void* out, int64_t ldo) {
  EpiParams ep{};
  ep.dependent = true;
  ep.out = out;
  ep.ldo = ldo;
  ep.remap.b = ep.remap.s = ep.remap.s_per_shard = 1;
  return ep;
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Workspaces of the products that may run with few rows: one after another in the forward.
size_t fc1_bytes(int64_t n, int64_t d, int64_t m, int t) {
  return gated_fc1_takes_few_rows(n, d, m, t) ? round256(gated_fc1_few_rows_workspace(n, d, m, t)) : 0;
}
size_t rows_bytes(int64_t n, int64_t cols, int64_t k) {
  return gemm_takes_few_rows(n, cols, k) ? round256(gemm_few_rows_workspace(n, cols, k)) : 0;
}

size_t dz_bytes(int64_t n, int64_t m) { return n <= 0 || m <= 0 ? 0 : (static_cast<size_t>(n) * m * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

size_t tpmlp_gated_forward_workspace_size(int64_t n, int64_t d, int64_t m, int t, tpmlp_dtype dt) {
  if (n <= 0 || check_gated_shape(n, d, m, t, TPMLP_GATE_SILU, dt) != TPMLP_OK) return 0;
  return fc1_bytes(n, d, m, t) + rows_bytes(n, d, m);
}

tpmlp_status tpmlp_gated_forward(const void* X, const void* A, const void* B, void* O, void* Z_save, void* Y_save,
                                 int64_t n, int64_t d, int64_t m, int t, int act, tpmlp_dtype dt, void* workspace,
                                 size_t ws_bytes, void* stream) {
  TPMLP_PASS(check_gated_shape(n, d, m, t, act, dt));
  TPMLP_PASS(check_ptrs({A, B}, 16, "pointers must be 16-byte aligned"));
  if (n == 0) return TPMLP_OK;
  TPMLP_PASS(check_ptrs({X, O, Y_save}, 16, "pointers must be 16-byte aligned"));
  if (!aligned(Z_save, 16)) return err(TPMLP_ERR_ALIGN, "pointers must be 16-byte aligned");
  const size_t need = tpmlp_gated_forward_workspace_size(n, d, m, t, dt);
  if (need > 0 && (!workspace || ws_bytes < need)) return err(TPMLP_ERR_WORKSPACE, "gated forward workspace too small");
  if (need > 0 && !aligned(workspace, 256)) return err(TPMLP_ERR_ALIGN, "workspace not 256-byte aligned");
  if (any_overlap({matrix(O, n, d), matrix(Z_save, n, 2 * m), matrix(Y_save, n, m),
                   flat_region(need ? workspace : nullptr, static_cast<int64_t>(need), 1)},
                  {matrix(X, n, d), matrix(A, d, 2 * m), matrix(B, m, d)}))
    return err(TPMLP_ERR_INVALID, "O, Z_save, Y_save or the workspace overlaps another tensor of the call");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool few = few_rows_allowed(), few1 = few && gated_fc1_takes_few_rows(n, d, m, t);
  if (few1) {
    TPMLP_PASS_CUDA(gated_fc1_few_rows(X, A, Z_save, Y_save, n, d, m, t, act, workspace, st, ctx), "gated FC1, few rows");
  } else {
    TPMLP_PASS_CUDA(gated_fc1_tc(X, A, Z_save, Y_save, n, d, m, t, act, st, ctx), "gated FC1 GEMM");
  }
  if (few && gemm_takes_few_rows(n, d, m)) {
    TPMLP_PASS_CUDA(gemm_few_rows(Y_save, B, true, O, n, d, m, static_cast<char*>(workspace) + fc1_bytes(n, d, m, t), true, st,
                                  ctx),
                    "gated FC2, few rows");
  } else {
    TPMLP_PASS_CUDA(gemm_bf16_tc(n, d, m, Operand{Y_save, n, m, m, false}, Operand{B, m, d, d, true}, kEpiStore, plain(O, d),
                                 st, ctx),
                    "gated FC2 GEMM");
  }
  return TPMLP_OK;
}

size_t tpmlp_gated_backward_workspace_size(int64_t n, int64_t d, int64_t m, tpmlp_dtype dt) {
  if (n <= 0 || check_gated_shape(n, d, m, 1, TPMLP_GATE_SILU, dt) != TPMLP_OK) return 0;
  return dz_bytes(n, m) + rows_bytes(n, d, 2 * m);
}

tpmlp_status tpmlp_gated_backward(const void* X, const void* A, const void* B, const void* G, const void* Z_save,
                                  const void* Y_save, void* dX, void* dA, void* dB, int64_t n, int64_t d, int64_t m, int t,
                                  int act, int wgrad, tpmlp_dtype dt, void* workspace, size_t ws_bytes, void* stream) {
  TPMLP_PASS(check_gated_shape(n, d, m, t, act, dt));
  if (wgrad != TPMLP_WGRAD_F32 && wgrad != TPMLP_WGRAD_F32_ADD && wgrad != TPMLP_WGRAD_OPERAND)
    return err(TPMLP_ERR_INVALID, "unknown form of the weights' gradients");
  TPMLP_PASS(check_ptrs({A, B, dA, dB}, 16, "pointers must be 16-byte aligned"));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t size = wgrad == TPMLP_WGRAD_OPERAND ? 2 : 4;
  if (any_overlap({matrix(dA, d, 2 * m, size), matrix(dB, m, d, size)}, {matrix(A, d, 2 * m), matrix(B, m, d)}))
    return err(TPMLP_ERR_INVALID, "dA or dB overlaps another tensor of the call");
  if (n == 0) {
    if (wgrad == TPMLP_WGRAD_F32_ADD) return TPMLP_OK;  // nothing to add
    TPMLP_PASS_CUDA(cudaMemsetAsync(dA, 0, static_cast<size_t>(size) * d * 2 * m, st), "zero dA");
    TPMLP_PASS_CUDA(cudaMemsetAsync(dB, 0, static_cast<size_t>(size) * m * d, st), "zero dB");
    return TPMLP_OK;
  }
  TPMLP_PASS(check_ptrs({X, G, Z_save, Y_save, dX}, 16, "pointers must be 16-byte aligned"));
  const size_t need = tpmlp_gated_backward_workspace_size(n, d, m, dt);
  if (!workspace || ws_bytes < need) return err(TPMLP_ERR_WORKSPACE, "gated backward workspace too small");
  if (!aligned(workspace, 256)) return err(TPMLP_ERR_ALIGN, "workspace not 256-byte aligned");
  if (any_overlap({matrix(dX, n, d), matrix(dA, d, 2 * m, size), matrix(dB, m, d, size),
                   flat_region(workspace, static_cast<int64_t>(need), 1)},
                  {matrix(X, n, d), matrix(A, d, 2 * m), matrix(B, m, d), matrix(G, n, d), matrix(Z_save, n, 2 * m),
                   matrix(Y_save, n, m)}))
    return err(TPMLP_ERR_INVALID, "dX, dA, dB or the workspace overlaps another tensor of the call");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  const EpiKind wepi = wgrad == TPMLP_WGRAD_OPERAND ? kEpiStore : wgrad == TPMLP_WGRAD_F32 ? kEpiStoreF32 : kEpiAccumF32;
  // D = [dY act'(Z_gate) Z_up | dY act(Z_gate)] shard by shard, laid out as Z
  TPMLP_PASS_CUDA(gated_dgrad1_tc(G, B, Z_save, workspace, n, d, m, t, act, st, ctx), "gated dgrad-1 GEMM");
  TPMLP_PASS_CUDA(gemm_bf16_twin(Product{m, d, Operand{Y_save, n, m, m, true}, Operand{G, n, d, d, true}, dB},
                                 Product{d, 2 * m, Operand{X, n, d, d, true}, Operand{workspace, n, 2 * m, 2 * m, true}, dA}, n,
                                 wepi, plain(nullptr, 0), st, ctx),
                  "gated wgrad GEMMs");
  // both projections' shares of dX are one sum over the 2 m columns of D
  if (few_rows_allowed() && gemm_takes_few_rows(n, d, 2 * m)) {
    TPMLP_PASS_CUDA(gemm_few_rows(workspace, A, false, dX, n, d, 2 * m, static_cast<char*>(workspace) + dz_bytes(n, m), true, st,
                                  ctx),
                    "gated dgrad-2, few rows");
    return TPMLP_OK;
  }
  TPMLP_PASS_CUDA(gemm_bf16_tc(n, d, 2 * m, Operand{workspace, n, 2 * m, 2 * m, false}, Operand{A, d, 2 * m, 2 * m, false},
                               kEpiStore, plain(dX, d), st, ctx),
                  "gated dgrad-2 GEMM");
  return TPMLP_OK;
}

}  // extern "C"

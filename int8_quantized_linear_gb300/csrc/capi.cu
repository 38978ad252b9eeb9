// C ABI of libi8ql.so: argument validation, per-device state and dispatch.
//
// Every entry point validates its arguments on the host before touching the
// CUDA runtime, so argument errors never launch anything and can be tested
// without a GPU.

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include <cmath>

#include "common.cuh"
#include "kv_schedule.cuh"
#include "kv_weights.cuh"
#include "rotary.cuh"

namespace i8ql {

// The sticky kernel-fault word; one instance per device context.
__device__ unsigned g_kernel_faults;

namespace {

constexpr int kMaxDevices = 64;

struct DeviceState {
    std::atomic<bool> ready{false};
    unsigned* err = nullptr;
    int sm_count = 0;
};

std::mutex g_mutex;
DeviceState g_devices[kMaxDevices];
std::atomic<int> g_debug_sk_timeout{0};
std::atomic<int> g_early_weights{0};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

i8ql_status check_k(int64_t K) {
    if (K <= 0) return I8QL_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > I8QL_MAX_K) return I8QL_ERR_UNSUPPORTED;
    return I8QL_OK;
}

i8ql_status check_rows(int64_t R) {
    if (R < 0) return I8QL_ERR_INVALID_ARG;
    if (R >= kMaxRows) return I8QL_ERR_UNSUPPORTED;
    return I8QL_OK;
}

i8ql_status check_matrix(const void* p, int64_t rows) {
    if (rows == 0) return I8QL_OK;
    if (p == nullptr || !aligned(p, 16)) return I8QL_ERR_INVALID_ARG;
    return I8QL_OK;
}

i8ql_status check_vec(const void* p, int64_t n, uintptr_t align) {
    if (n == 0) return I8QL_OK;
    if (p == nullptr || !aligned(p, align)) return I8QL_ERR_INVALID_ARG;
    return I8QL_OK;
}

#define I8QL_TRY(expr)                       \
    do {                                     \
        i8ql_status _s = (expr);             \
        if (_s != I8QL_OK) return _s;        \
    } while (0)

i8ql_status from_cuda(cudaError_t e) { return e == cudaSuccess ? I8QL_OK : I8QL_ERR_CUDA; }

}  // namespace

bool debug_sk_timeout() { return g_debug_sk_timeout.load(std::memory_order_relaxed) != 0; }
bool early_weight_loads() { return g_early_weights.load(std::memory_order_relaxed) != 0; }

bool launch_env(void* stream, LaunchEnv* env, i8ql_status* status) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        *status = I8QL_ERR_NO_DEVICE;
        return false;
    }
    DeviceState& st = g_devices[dev];
    if (!st.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (!st.ready.load(std::memory_order_relaxed)) {
            int major = 0, minor = 0, sms = 0;
            if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
                cudaGetLastError();
                *status = I8QL_ERR_CUDA;
                return false;
            }
            if (major != 10 || minor != 3) {
                *status = I8QL_ERR_NO_DEVICE;
                return false;
            }
            void* addr = nullptr;
            if (cudaGetSymbolAddress(&addr, g_kernel_faults) != cudaSuccess) {
                cudaGetLastError();
                *status = I8QL_ERR_CUDA;
                return false;
            }
            st.err = static_cast<unsigned*>(addr);
            st.sm_count = sms;
            st.ready.store(true, std::memory_order_release);
        }
    }
    env->stream = static_cast<cudaStream_t>(stream);
    env->err = st.err;
    env->sm_count = st.sm_count;
    return true;
}

}  // namespace i8ql

using namespace i8ql;

extern "C" {

i8ql_status quantize_weight_per_channel_int8(const i8ql_bf16* w, int64_t N, int64_t K, int8_t* q,
                                             float* scale, void* stream) {
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_k(K));
    I8QL_TRY(check_matrix(w, N));
    I8QL_TRY(check_matrix(q, N));
    I8QL_TRY(check_vec(scale, N, 4));
    if (N == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_quant_rows(w, N, K, q, nullptr, scale, env));
}

i8ql_status quantize_act_per_token_int8(const i8ql_bf16* x, int64_t M, int64_t K, int8_t* q,
                                        float* scale, void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    I8QL_TRY(check_matrix(x, M));
    I8QL_TRY(check_matrix(q, M));
    I8QL_TRY(check_vec(scale, M, 4));
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_quant_rows(x, M, K, q, nullptr, scale, env));
}

i8ql_status w8a8_gemm(const int8_t* qx, const float* sx, const int8_t* qw, const float* sw,
                      const i8ql_bf16* bias, i8ql_bf16* y, int32_t* acc_debug, int64_t M, int64_t N,
                      int64_t K, void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(qx, M));
    I8QL_TRY(check_vec(sx, M, 4));
    I8QL_TRY(check_matrix(qw, N));
    I8QL_TRY(check_vec(sw, N, 4));
    if (bias != nullptr && !aligned(bias, 2)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(y, M));
    if (acc_debug != nullptr && !aligned(acc_debug, 16)) return I8QL_ERR_INVALID_ARG;
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w8a8(qx, sx, qw, sw, bias, y, acc_debug, M, N, K, env));
}

i8ql_status w8a8_linear(const i8ql_bf16* x, const int8_t* qw, const float* sw, const i8ql_bf16* bias,
                        i8ql_bf16* y, int8_t* qx, float* sx, int32_t* acc_debug, int64_t M, int64_t N, int64_t K,
                        void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(x, M));
    I8QL_TRY(check_matrix(qw, N));
    I8QL_TRY(check_vec(sw, N, 4));
    if (bias != nullptr && !aligned(bias, 2)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(y, M));
    if (qx != nullptr) I8QL_TRY(check_matrix(qx, M));
    if (sx != nullptr && !aligned(sx, 4)) return I8QL_ERR_INVALID_ARG;
    if (acc_debug != nullptr && !aligned(acc_debug, 16)) return I8QL_ERR_INVALID_ARG;
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w8a8_linear(x, qw, sw, bias, y, qx, sx, acc_debug, M, N, K, env));
}

i8ql_status w8a8_linear_fused(const i8ql_bf16* x, const int8_t* qw, const float* sw, const i8ql_bf16* bias,
                              i8ql_bf16* y, int8_t* qx, float* sx, int32_t* acc_debug, int64_t M, int64_t N, int64_t K,
                              void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    if (M > kW8A8FusedMaxM) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(x, M));
    I8QL_TRY(check_matrix(qw, N));
    I8QL_TRY(check_vec(sw, N, 4));
    if (bias != nullptr && !aligned(bias, 2)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(y, M));
    if (qx != nullptr) I8QL_TRY(check_matrix(qx, M));
    if (sx != nullptr && !aligned(sx, 4)) return I8QL_ERR_INVALID_ARG;
    if (acc_debug != nullptr && !aligned(acc_debug, 16)) return I8QL_ERR_INVALID_ARG;
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w8a8_decode_fused(x, qw, sw, bias, y, qx, sx, acc_debug, M, N, K, env));
}

i8ql_status w8a16_gemm(const i8ql_bf16* x, const int8_t* qw, const float* sw, i8ql_bf16* y,
                       int64_t M, int64_t N, int64_t K, void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(x, M));
    I8QL_TRY(check_matrix(qw, N));
    I8QL_TRY(check_vec(sw, N, 4));
    I8QL_TRY(check_matrix(y, M));
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w8a16(x, nullptr, 1, qw, sw, y, M, N, K, env));
}

i8ql_status grouped_w8a16_gemm(const i8ql_bf16* x, const int32_t* offsets, int64_t E,
                               const int8_t* qw, const float* sw, i8ql_bf16* y, int64_t T_total,
                               int64_t N, int64_t K, void* stream) {
    I8QL_TRY(check_rows(T_total));
    I8QL_TRY(check_k(K));
    if (N <= 0 || E <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    if (E > 65535) return I8QL_ERR_UNSUPPORTED;
    if ((double)E * (double)N * (double)K > 9.0e18) return I8QL_ERR_UNSUPPORTED;
    if (offsets == nullptr || !aligned(offsets, 4)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(x, T_total));
    if (qw == nullptr || !aligned(qw, 16)) return I8QL_ERR_INVALID_ARG;
    if (sw == nullptr || !aligned(sw, 4)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(y, T_total));
    if (T_total == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w8a16(x, offsets, E, qw, sw, y, T_total, N, K, env));
}

i8ql_status quantize_weight_per_channel_fp8(const i8ql_bf16* w, int64_t N, int64_t K, uint8_t* q, float* scale,
                                            void* stream) {
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_k(K));
    I8QL_TRY(check_matrix(w, N));
    I8QL_TRY(check_matrix(q, N));
    I8QL_TRY(check_vec(scale, N, 4));
    if (N == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_quant_rows_fp8(w, N, K, q, scale, env));
}

i8ql_status quantize_act_per_token_fp8(const i8ql_bf16* x, int64_t M, int64_t K, uint8_t* q, float* scale,
                                       void* stream) {
    return quantize_weight_per_channel_fp8(x, M, K, q, scale, stream);
}

i8ql_status w8a8_fp8_gemm(const uint8_t* qx, const float* sx, const uint8_t* qw, const float* sw,
                          const i8ql_bf16* bias, i8ql_bf16* y, int64_t M, int64_t N, int64_t K, void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(qx, M));
    I8QL_TRY(check_vec(sx, M, 4));
    I8QL_TRY(check_matrix(qw, N));
    I8QL_TRY(check_vec(sw, N, 4));
    if (bias != nullptr && !aligned(bias, 2)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(y, M));
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_fp8_gemm(qx, sx, qw, sw, bias, y, M, N, K, env));
}

i8ql_status w8a8_fp8_linear(const i8ql_bf16* x, const uint8_t* qw, const float* sw, const i8ql_bf16* bias,
                            i8ql_bf16* y, uint8_t* qx, float* sx, int64_t M, int64_t N, int64_t K, void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(x, M));
    I8QL_TRY(check_matrix(qw, N));
    I8QL_TRY(check_vec(sw, N, 4));
    if (bias != nullptr && !aligned(bias, 2)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(y, M));
    if (qx != nullptr) I8QL_TRY(check_matrix(qx, M));
    if (sx != nullptr && !aligned(sx, 4)) return I8QL_ERR_INVALID_ARG;
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_fp8_linear(x, qw, sw, bias, y, qx, sx, M, N, K, env));
}

i8ql_status quantize_weight_w4_g128(const i8ql_bf16* w, int64_t N, int64_t K, uint8_t* q, i8ql_bf16* scale,
                                    void* stream) {
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_k(K));
    if (K % 128 != 0) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_matrix(w, N));
    I8QL_TRY(check_matrix(q, N));
    I8QL_TRY(check_vec(scale, N, 2));
    if (N == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_quant_w4(w, N, K, q, scale, env));
}

i8ql_status w4a16_gemm(const i8ql_bf16* x, const uint8_t* q, const i8ql_bf16* scale, i8ql_bf16* y, int64_t M,
                       int64_t N, int64_t K, void* stream) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (K % 128 != 0) return I8QL_ERR_UNSUPPORTED;
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    I8QL_TRY(check_matrix(x, M));
    I8QL_TRY(check_matrix(q, N));
    I8QL_TRY(check_vec(scale, N, 2));
    I8QL_TRY(check_matrix(y, M));
    if (M == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w4a16(x, q, scale, y, M, N, K, env));
}

i8ql_status moe_route_topk(const float* logits, int64_t T, int64_t E, int64_t top_k, int64_t n_shared,
                           int32_t* offsets, int32_t* row_token, int32_t* token_row, float* slot_weight,
                           void* stream) {
    if (T < 0 || E <= 0 || top_k <= 0 || top_k > E || n_shared < 0) return I8QL_ERR_INVALID_ARG;
    if (E > 256 || n_shared > 64 || T > 65535 || moe_route_smem(T, E) == kRouteTooLarge)
        return I8QL_ERR_UNSUPPORTED;
    if (offsets == nullptr || !aligned(offsets, 4)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_vec(logits, T, 4));
    I8QL_TRY(check_vec(row_token, T, 4));
    I8QL_TRY(check_vec(token_row, T, 4));
    I8QL_TRY(check_vec(slot_weight, T, 4));
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_moe_route(logits, T, E, top_k, n_shared, offsets, row_token, token_row, slot_weight, env));
}

i8ql_status grouped_w8a16_silu_mul(const i8ql_bf16* x, const int32_t* row_token, const int32_t* offsets, int64_t E,
                                   const int8_t* qw, const float* sw, i8ql_bf16* h, int64_t T_total, int64_t I,
                                   int64_t K, void* stream) {
    I8QL_TRY(check_rows(T_total));
    I8QL_TRY(check_k(K));
    if (I <= 0 || E <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(2 * I));
    if (E > 65535) return I8QL_ERR_UNSUPPORTED;
    if ((double)E * (double)(2 * I) * (double)K > 9.0e18) return I8QL_ERR_UNSUPPORTED;
    if (offsets == nullptr || !aligned(offsets, 4)) return I8QL_ERR_INVALID_ARG;
    if (row_token != nullptr && !aligned(row_token, 4)) return I8QL_ERR_INVALID_ARG;
    if (x == nullptr && T_total > 0) return I8QL_ERR_INVALID_ARG;
    if (x != nullptr && !aligned(x, 16)) return I8QL_ERR_INVALID_ARG;
    if (qw == nullptr || !aligned(qw, 16)) return I8QL_ERR_INVALID_ARG;
    if (sw == nullptr || !aligned(sw, 4)) return I8QL_ERR_INVALID_ARG;
    if (T_total > 0 && (h == nullptr || !aligned(h, 2))) return I8QL_ERR_INVALID_ARG;
    if (T_total == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_w8a16(x, offsets, E, qw, sw, h, T_total, 2 * I, K, env, row_token, I));
}

i8ql_status moe_combine(const i8ql_bf16* yd, const int32_t* token_row, const float* slot_weight, i8ql_bf16* out,
                        int64_t T, int64_t S, int64_t H, void* stream) {
    if (T < 0 || S <= 0 || H <= 0) return I8QL_ERR_INVALID_ARG;
    if (H % 8 != 0 || T > 65535) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_vec(token_row, T, 4));
    I8QL_TRY(check_vec(slot_weight, T, 4));
    I8QL_TRY(check_matrix(yd, T));
    I8QL_TRY(check_matrix(out, T));
    if (T == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_moe_combine(yd, token_row, slot_weight, out, T, S, H, env));
}

i8ql_status moe_expert_mlp_w8a16(const i8ql_bf16* x, const float* logits, int64_t E_routed, int64_t top_k,
                                 int64_t n_shared, const int8_t* qw_gate_up, const float* sw_gate_up,
                                 const int8_t* qw_down, const float* sw_down, i8ql_bf16* out, int64_t T, int64_t H,
                                 int64_t I, void* stream) {
    if (T < 0 || E_routed <= 0 || top_k <= 0 || top_k > E_routed || n_shared < 0 || H <= 0 || I <= 0)
        return I8QL_ERR_INVALID_ARG;
    if (E_routed > 256 || n_shared > 64 || T > 65535 || moe_route_smem(T, E_routed) == kRouteTooLarge)
        return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_k(H));
    I8QL_TRY(check_k(I));
    I8QL_TRY(check_matrix(x, T));
    I8QL_TRY(check_vec(logits, T, 4));
    I8QL_TRY(check_matrix(out, T));
    if (qw_gate_up == nullptr || !aligned(qw_gate_up, 16) || qw_down == nullptr || !aligned(qw_down, 16))
        return I8QL_ERR_INVALID_ARG;
    if (sw_gate_up == nullptr || !aligned(sw_gate_up, 4) || sw_down == nullptr || !aligned(sw_down, 4))
        return I8QL_ERR_INVALID_ARG;
    if (T == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_moe_mlp(x, logits, E_routed, top_k, n_shared, qw_gate_up, sw_gate_up, qw_down, sw_down,
                                    out, T, H, I, env));
}

namespace {

// Sizes every call on the key/value cache checks.
i8ql_status check_kv(int64_t H, int64_t D, int64_t bits, int64_t page_size, int64_t num_pages) {
    if (H <= 0 || D <= 0 || num_pages <= 0 || page_size <= 0) return I8QL_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || (bits != 4 && bits != 8) || H > 65535 || num_pages >= kMaxRows ||
        page_size < kKvMinPage || page_size > kKvMaxPage || (page_size & (page_size - 1)) != 0)
        return I8QL_ERR_UNSUPPORTED;
    return I8QL_OK;
}

// Token rows of n values, `stride` elements apart.
i8ql_status check_strided(const void* p, int64_t rows, int64_t n, int64_t stride) {
    if (stride < n || stride % 8 != 0) return I8QL_ERR_INVALID_ARG;
    return check_matrix(p, rows);
}

KvCache make_kv_cache(const uint8_t* codes, const i8ql_bf16* params, int64_t H, int64_t page_size, int64_t num_pages) {
    KvCache c;
    c.codes = const_cast<uint8_t*>(codes);
    c.params = reinterpret_cast<uint32_t*>(const_cast<i8ql_bf16*>(params));
    c.pages = num_pages;
    c.H = (int)H;
    c.page_shift = 0;
    while (((int64_t)1 << c.page_shift) < page_size) ++c.page_shift;
    return c;
}

i8ql_status check_kv_attention(int64_t B, int64_t T_q, int64_t Hq, int64_t H, int64_t page_size, int64_t table_width,
                               int64_t max_q) {
    if (B < 0 || T_q < 0 || Hq <= 0 || Hq % H != 0 || table_width <= 0 || max_q < 0 || (max_q == 0 && T_q > 0))
        return I8QL_ERR_INVALID_ARG;
    if (B >= kMaxRows || Hq > 65535 || T_q >= ((int64_t)1 << 30) || T_q * (Hq / H) >= ((int64_t)1 << 30) ||
        table_width > (kMaxRows - 65536) / page_size)
        return I8QL_ERR_UNSUPPORTED;
    return I8QL_OK;
}

}  // namespace

i8ql_status kv_cache_store(const i8ql_bf16* k, const i8ql_bf16* v, int64_t k_stride, int64_t v_stride,
                           const int64_t* slots, uint8_t* codes, i8ql_bf16* params, int64_t T, int64_t H, int64_t D,
                           int64_t bits, int64_t page_size, int64_t num_pages, void* stream) {
    I8QL_TRY(check_rows(T));
    I8QL_TRY(check_kv(H, D, bits, page_size, num_pages));
    if (T * H >= ((int64_t)1 << 30)) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_strided(k, T, H * D, k_stride));
    I8QL_TRY(check_strided(v, T, H * D, v_stride));
    I8QL_TRY(check_vec(slots, T, 8));
    I8QL_TRY(check_matrix(codes, T));
    I8QL_TRY(check_matrix(params, T));
    if (T == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_kv_store(k, v, k_stride, v_stride, slots, make_kv_cache(codes, params, H, page_size, num_pages),
                                     T, D, bits, env));
}

i8ql_status kv_cache_load(const uint8_t* codes, const i8ql_bf16* params, const int64_t* slots, i8ql_bf16* k,
                          i8ql_bf16* v, int64_t T, int64_t H, int64_t D, int64_t bits, int64_t page_size,
                          int64_t num_pages, void* stream) {
    I8QL_TRY(check_rows(T));
    I8QL_TRY(check_kv(H, D, bits, page_size, num_pages));
    if (T * H >= ((int64_t)1 << 30)) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_vec(slots, T, 8));
    I8QL_TRY(check_matrix(codes, T));
    I8QL_TRY(check_matrix(params, T));
    I8QL_TRY(check_matrix(k, T));
    I8QL_TRY(check_matrix(v, T));
    if (T == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_kv_load(make_kv_cache(codes, params, H, page_size, num_pages), slots, k, v, T, D, bits, env));
}

i8ql_status i8ql_kv_attention_workspace(int64_t B, int64_t T_q, int64_t Hq, int64_t H, int64_t D, int64_t bits,
                                        int64_t page_size, int64_t table_width, int64_t max_q, int64_t* bytes) {
    I8QL_TRY(check_kv(H, D, bits, page_size, 1));
    I8QL_TRY(check_kv_attention(B, T_q, Hq, H, page_size, table_width, max_q));
    if (bytes == nullptr) return I8QL_ERR_INVALID_ARG;
    *bytes = 0;
    if (B == 0 || T_q == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(nullptr, &env, &s)) return s;
    *bytes = (int64_t)kv_attention_workspace(B, T_q, Hq / H, H, D, bits, table_width * page_size, max_q, env.sm_count);
    return I8QL_OK;
}

i8ql_status kv_cache_attention(const i8ql_bf16* q, int64_t q_stride, const uint8_t* codes, const i8ql_bf16* params,
                               const int32_t* page_table, int64_t table_width, const int32_t* kv_lens,
                               const int32_t* q_offsets, i8ql_bf16* out, int64_t B, int64_t T_q, int64_t Hq, int64_t H,
                               int64_t D, int64_t bits, int64_t page_size, int64_t num_pages, int64_t max_q,
                               int64_t window, float softmax_scale, void* workspace, int64_t workspace_bytes,
                               void* stream) {
    I8QL_TRY(check_kv(H, D, bits, page_size, num_pages));
    I8QL_TRY(check_kv_attention(B, T_q, Hq, H, page_size, table_width, max_q));
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (window < 0 || !std::isfinite(scale_log2)) return I8QL_ERR_INVALID_ARG;
    if (q_offsets == nullptr && T_q != B) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_strided(q, T_q, Hq * D, q_stride));
    I8QL_TRY(check_matrix(codes, T_q));
    I8QL_TRY(check_matrix(params, T_q));
    I8QL_TRY(check_vec(page_table, T_q, 4));
    I8QL_TRY(check_vec(kv_lens, T_q, 4));
    if (q_offsets != nullptr && !aligned(q_offsets, 4)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(out, T_q));
    if (T_q == 0) return I8QL_OK;
    if (B == 0) return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    const int64_t G = Hq / H;
    const int64_t need =
        (int64_t)kv_attention_workspace(B, T_q, G, H, D, bits, table_width * page_size, max_q, env.sm_count);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need) return I8QL_ERR_WORKSPACE_LIMIT;
        if (!aligned(workspace, 16)) return I8QL_ERR_INVALID_ARG;
    }
    KvAttnParams p = {};
    p.cache = make_kv_cache(codes, params, H, page_size, num_pages);
    p.q = q;
    p.q_stride = q_stride;
    p.table = page_table;
    p.table_width = table_width;
    p.kv_lens = kv_lens;
    p.q_offsets = q_offsets;
    p.out = out;
    p.B = B;
    p.T_q = T_q;
    p.G = (int)G;
    p.window = window;
    p.scale_log2 = scale_log2;
    p.err = env.err;
    return from_cuda(launch_kv_attention(p, D, bits, max_q, workspace, env));
}

namespace {

// Whether token rows of a_n values at `a` and of b_n at `b` (`rows` of them, their strides
// apart) share memory.
bool meet(const i8ql_bf16* a, int64_t a_stride, int64_t a_n, const i8ql_bf16* b, int64_t b_stride, int64_t b_n,
          int64_t rows) {
    if (b < a) return meet(b, b_stride, b_n, a, a_stride, a_n, rows);
    const int64_t apart = b - a;
    if (apart >= (rows - 1) * a_stride + a_n) return false;
    if (a_stride != b_stride) return true;
    // (neighbours in rows of the same width do not meet)
    return apart % a_stride < a_n || apart % a_stride > a_stride - b_n;
}

// The same, but for the very same rows.
bool tangled(const i8ql_bf16* a, int64_t a_stride, const i8ql_bf16* b, int64_t b_stride, int64_t rows, int64_t n) {
    if (a == b) return a_stride != b_stride && rows > 1;
    return meet(a, a_stride, n, b, b_stride, n, rows);
}

// A table of angles for T tokens' rows of D channels.
i8ql_status check_rotary(const float* table, int64_t table_rows, const int64_t* positions, int64_t T, int64_t D,
                         int64_t rot, int64_t multiple, int32_t interleaved) {
    if (rot <= 0 || table_rows < 0 || (interleaved != 0 && interleaved != 1)) return I8QL_ERR_INVALID_ARG;
    if (rot > D || rot % multiple != 0 || table_rows >= kMaxRows) return I8QL_ERR_UNSUPPORTED;
    if (T == 0) return I8QL_OK;
    if (positions == nullptr && table_rows < T) return I8QL_ERR_INVALID_ARG;
    if (positions != nullptr && !aligned(positions, 8)) return I8QL_ERR_INVALID_ARG;
    return check_matrix(table, table_rows);
}

RotaryTable make_rotary(const float* table, int64_t table_rows, const int64_t* positions, int64_t rot) {
    RotaryTable t;
    t.rows = table;
    t.count = table_rows;
    t.positions = positions;
    t.rot = (int)rot;
    return t;
}

}  // namespace

i8ql_status rotary_table(const double* freqs, const int64_t* positions, float* table, int64_t P, int64_t F,
                         float amplitude, void* stream) {
    I8QL_TRY(check_rows(P));
    if (F <= 0 || !std::isfinite(amplitude)) return I8QL_ERR_INVALID_ARG;
    if (F > I8QL_ROTARY_MAX_D / 2) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_vec(freqs, P, 8));
    if (positions != nullptr && !aligned(positions, 8)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(table, P));
    if (P == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_rotary_table(freqs, positions, table, P, F, amplitude, env));
}

i8ql_status rotary_apply(const i8ql_bf16* x, int64_t x_stride, const float* table, int64_t table_rows,
                         const int64_t* positions, i8ql_bf16* out, int64_t out_stride, int64_t T, int64_t heads,
                         int64_t D, int64_t rot, int32_t interleaved, int32_t backward, void* stream) {
    I8QL_TRY(check_rows(T));
    if (heads <= 0 || D <= 0 || (backward != 0 && backward != 1)) return I8QL_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > I8QL_ROTARY_MAX_D || heads > 65535 || T * heads >= ((int64_t)1 << 30))
        return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_rotary(table, table_rows, positions, T, D, rot, 8, interleaved));
    I8QL_TRY(check_strided(x, T, heads * D, x_stride));
    I8QL_TRY(check_strided(out, T, heads * D, out_stride));
    if (T == 0) return I8QL_OK;
    if (tangled(x, x_stride, out, out_stride, T, heads * D)) return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_rotary_apply(x, x_stride, make_rotary(table, table_rows, positions, rot), out, out_stride, T,
                                         heads, D, interleaved != 0, backward != 0, env));
}

i8ql_status kv_cache_store_rotary(const i8ql_bf16* q, int64_t q_stride, i8ql_bf16* q_out, int64_t q_out_stride,
                                  const i8ql_bf16* k, const i8ql_bf16* v, int64_t k_stride, int64_t v_stride,
                                  const float* table, int64_t table_rows, const int64_t* positions,
                                  const int64_t* slots, uint8_t* codes, i8ql_bf16* params, int64_t T, int64_t Hq,
                                  int64_t H, int64_t D, int64_t bits, int64_t page_size, int64_t num_pages, int64_t rot,
                                  int32_t interleaved, void* stream) {
    I8QL_TRY(check_rows(T));
    I8QL_TRY(check_kv(H, D, bits, page_size, num_pages));
    if (Hq < 0) return I8QL_ERR_INVALID_ARG;
    if (Hq > 65535 || T * (Hq + H) >= ((int64_t)1 << 30)) return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_rotary(table, table_rows, positions, T, D, rot, 16, interleaved));
    if (Hq > 0) {
        I8QL_TRY(check_strided(q, T, Hq * D, q_stride));
        I8QL_TRY(check_strided(q_out, T, Hq * D, q_out_stride));
    }
    I8QL_TRY(check_strided(k, T, H * D, k_stride));
    I8QL_TRY(check_strided(v, T, H * D, v_stride));
    I8QL_TRY(check_vec(slots, T, 8));
    I8QL_TRY(check_matrix(codes, T));
    I8QL_TRY(check_matrix(params, T));
    if (T == 0) return I8QL_OK;
    if (Hq > 0 && (tangled(q, q_stride, q_out, q_out_stride, T, Hq * D) ||
                   meet(q_out, q_out_stride, Hq * D, k, k_stride, H * D, T) ||
                   meet(q_out, q_out_stride, Hq * D, v, v_stride, H * D, T)))
        return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    return from_cuda(launch_kv_store_rotary(q, q_stride, q_out, q_out_stride, k, v, k_stride, v_stride,
                                            make_rotary(table, table_rows, positions, rot), interleaved != 0, slots,
                                            make_kv_cache(codes, params, H, page_size, num_pages), T, Hq, D, bits, env));
}

namespace {

// What kv_cache_weights needs of workspace.  max_q is held to the query tokens there are: fewer rows can
// mean a finer split of the tokens, so a bound above them would tell another size.
int64_t weights_workspace(int64_t B, int64_t T_q, int64_t Hq, int64_t H, int64_t max_kv, int64_t& max_q, const LaunchEnv& env) {
    max_q = max_q < T_q ? max_q : T_q;
    return (int64_t)kv_weights_workspace(B, T_q, Hq / H, H, max_kv, max_q, env.sm_count);
}

}  // namespace

i8ql_status i8ql_kv_weights_workspace(int64_t B, int64_t T_q, int64_t Hq, int64_t H, int64_t D, int64_t bits,
                                      int64_t page_size, int64_t table_width, int64_t max_q, int64_t* bytes) {
    I8QL_TRY(check_kv(H, D, bits, page_size, 1));
    I8QL_TRY(check_kv_attention(B, T_q, Hq, H, page_size, table_width, max_q));
    if (bytes == nullptr) return I8QL_ERR_INVALID_ARG;
    *bytes = 0;
    if (B == 0 || T_q == 0) return I8QL_OK;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(nullptr, &env, &s)) return s;
    *bytes = weights_workspace(B, T_q, Hq, H, table_width * page_size, max_q, env);
    return I8QL_OK;
}

i8ql_status kv_cache_weights(const i8ql_bf16* q, int64_t q_stride, const uint8_t* codes, const i8ql_bf16* params,
                             const int32_t* page_table, int64_t table_width, const int32_t* kv_lens,
                             const int32_t* q_offsets, const float* previous, float* weights, int64_t B, int64_t T_q,
                             int64_t Hq, int64_t H, int64_t D, int64_t bits, int64_t page_size, int64_t num_pages,
                             int64_t max_q, int64_t window, float softmax_scale, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    I8QL_TRY(check_kv(H, D, bits, page_size, num_pages));
    I8QL_TRY(check_kv_attention(B, T_q, Hq, H, page_size, table_width, max_q));
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (window < 0 || !std::isfinite(scale_log2)) return I8QL_ERR_INVALID_ARG;
    if (q_offsets == nullptr && T_q != B) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_strided(q, T_q, Hq * D, q_stride));
    I8QL_TRY(check_matrix(codes, T_q));
    I8QL_TRY(check_matrix(params, T_q));
    I8QL_TRY(check_vec(page_table, T_q, 4));
    I8QL_TRY(check_vec(kv_lens, T_q, 4));
    if (q_offsets != nullptr && !aligned(q_offsets, 4)) return I8QL_ERR_INVALID_ARG;
    if (previous != nullptr && !aligned(previous, 16)) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_matrix(weights, T_q));
    if (T_q == 0) return I8QL_OK;
    if (B == 0) return I8QL_ERR_INVALID_ARG;
    // (previous weights are read while others are written: the same, or apart)
    const int64_t places = num_pages * H * page_size;
    if (previous != nullptr && previous != weights && previous < weights + places && weights < previous + places)
        return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    const int64_t G = Hq / H, max_kv = table_width * page_size;
    const int64_t need = weights_workspace(B, T_q, Hq, H, max_kv, max_q, env);
    if (!kv_weights_fits(B, G, H, max_kv, max_q, env.sm_count)) return I8QL_ERR_UNSUPPORTED;
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need) return I8QL_ERR_WORKSPACE_LIMIT;
        if (!aligned(workspace, 16)) return I8QL_ERR_INVALID_ARG;
    }
    KvWeightsParams p = {};
    p.a.cache = make_kv_cache(codes, params, H, page_size, num_pages);
    p.a.q = q;
    p.a.q_stride = q_stride;
    p.a.table = page_table;
    p.a.table_width = table_width;
    p.a.kv_lens = kv_lens;
    p.a.q_offsets = q_offsets;
    p.a.B = B;
    p.a.T_q = T_q;
    p.a.G = (int)G;
    p.a.window = window;
    p.a.scale_log2 = scale_log2;
    p.a.err = env.err;
    p.max_q = max_q;
    p.previous = previous;
    p.weights = weights;
    return from_cuda(launch_kv_weights(p, D, bits, workspace, env));
}

i8ql_status kv_cache_evict(uint8_t* codes, i8ql_bf16* params, float* weights, const int32_t* page_table,
                           int64_t table_width, const int32_t* kv_lens, const int32_t* new_table, int64_t new_width,
                           int32_t* new_lens, int32_t* kept, int64_t B, int64_t H, int64_t D, int64_t bits,
                           int64_t page_size, int64_t num_pages, int64_t budget, int64_t first, int64_t last,
                           void* stream) {
    I8QL_TRY(check_kv(H, D, bits, page_size, num_pages));
    if (B < 0 || table_width <= 0 || budget <= 0 || first < 0 || last < 0 || first > budget || last > budget - first)
        return I8QL_ERR_INVALID_ARG;
    if (new_table == nullptr) {
        new_table = page_table;
        new_width = table_width;
    }
    if (new_width <= 0 || (new_table == page_table && new_width != table_width)) return I8QL_ERR_INVALID_ARG;
    if (B >= kMaxRows || table_width > (kMaxRows - 65536) / page_size || new_width > (kMaxRows - 65536) / page_size ||
        budget > kMaxRows - 65536 || !kv_evict_fits(B, H, D * bits / 8, budget))
        return I8QL_ERR_UNSUPPORTED;
    I8QL_TRY(check_matrix(codes, B));
    I8QL_TRY(check_matrix(params, B));
    I8QL_TRY(check_matrix(weights, B));
    I8QL_TRY(check_vec(page_table, B, 4));
    I8QL_TRY(check_vec(new_table, B, 4));
    I8QL_TRY(check_vec(kv_lens, B, 4));
    I8QL_TRY(check_vec(new_lens, B, 4));
    I8QL_TRY(check_vec(kept, B, 4));
    if (B == 0) return I8QL_OK;
    // (every head reads kv_lens while the first writes new_lens)
    if (new_lens < kv_lens + B && kv_lens < new_lens + B) return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    KvEvictParams p = {};
    p.cache = make_kv_cache(codes, params, H, page_size, num_pages);
    p.weights = weights;
    p.table = page_table;
    p.table_width = table_width;
    p.kv_lens = kv_lens;
    p.new_table = new_table;
    p.new_width = new_width;
    p.new_lens = new_lens;
    p.kept = kept;
    p.B = B;
    p.budget = (int)budget;
    p.first = (int)first;
    p.last = (int)last;
    p.row_bytes = (int)(D * bits / 8);
    p.err = env.err;
    return from_cuda(launch_kv_evict(p, env));
}

i8ql_status i8ql_get_device_error(void* stream) {
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(stream, &env, &s)) return s;
    if (cudaStreamSynchronize(env.stream) != cudaSuccess) return I8QL_ERR_CUDA;
    unsigned word = 0;
    if (cudaMemcpy(&word, env.err, sizeof word, cudaMemcpyDeviceToHost) != cudaSuccess)
        return I8QL_ERR_CUDA;
    if (word != 0) {
        const unsigned zero = 0;
        if (cudaMemcpy(env.err, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
            return I8QL_ERR_CUDA;
    }
    if (word & kErrBitTimeout) return I8QL_ERR_TIMEOUT;
    if (word & kErrBitBadOffsets) return I8QL_ERR_BAD_OFFSETS;
    if (word & kErrBitBadIndex) return I8QL_ERR_BAD_INDEX;
    return I8QL_OK;
}

namespace {

i8ql_status plan_query(int64_t M, int64_t N, int64_t K, bool allow_sk, int32_t* tile_n, int32_t* split_k,
                       int32_t* cta_pair) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    if (tile_n == nullptr || split_k == nullptr || cta_pair == nullptr) return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(nullptr, &env, &s)) return s;
    int bn = 0, split = 0, pair = 0;
    I8QL_TRY(from_cuda(w8a8_plan(M, N, K, env.sm_count, allow_sk, &bn, &split, &pair)));
    *tile_n = bn;
    *split_k = split;
    *cta_pair = pair;
    return I8QL_OK;
}

}  // namespace

i8ql_status i8ql_w8a8_plan(int64_t M, int64_t N, int64_t K, int32_t* tile_n, int32_t* split_k, int32_t* cta_pair) {
    return plan_query(M, N, K, true, tile_n, split_k, cta_pair);
}

i8ql_status i8ql_w8a8_noalloc_plan(int64_t M, int64_t N, int64_t K, int32_t* tile_n, int32_t* split_k,
                                   int32_t* cta_pair) {
    return plan_query(M, N, K, false, tile_n, split_k, cta_pair);
}

i8ql_status i8ql_w8a8_linear_launches(int64_t M, int64_t N, int64_t K, int32_t* launches) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    if (launches == nullptr) return I8QL_ERR_INVALID_ARG;
    if (M == 0) {
        *launches = 0;
        return I8QL_OK;
    }
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(nullptr, &env, &s)) return s;
    *launches = w8a8_linear_one_launch(M, N, K, env.sm_count) ? 1 : 2;
    return I8QL_OK;
}

i8ql_status i8ql_fp8_plan(int64_t M, int64_t N, int64_t K, int32_t* tile_n, int32_t* split_k, int32_t* cta_pair) {
    I8QL_TRY(check_rows(M));
    I8QL_TRY(check_k(K));
    if (N <= 0) return I8QL_ERR_INVALID_ARG;
    I8QL_TRY(check_rows(N));
    if (tile_n == nullptr || split_k == nullptr || cta_pair == nullptr) return I8QL_ERR_INVALID_ARG;
    LaunchEnv env;
    i8ql_status s;
    if (!launch_env(nullptr, &env, &s)) return s;
    int bn = 0, split = 0, pair = 0;
    I8QL_TRY(from_cuda(fp8_plan(M, N, K, env.sm_count, &bn, &split, &pair)));
    *tile_n = bn;
    *split_k = split;
    *cta_pair = pair;
    return I8QL_OK;
}

const char* i8ql_status_string(i8ql_status status) {
    switch (status) {
        case I8QL_OK: return "ok";
        case I8QL_ERR_INVALID_ARG: return "invalid argument (null, negative size or misaligned pointer)";
        case I8QL_ERR_UNSUPPORTED: return "unsupported size (K must be a positive multiple of 16, at most 133144)";
        case I8QL_ERR_CUDA: return "CUDA runtime or launch failure";
        case I8QL_ERR_TIMEOUT: return "a kernel's bounded wait timed out";
        case I8QL_ERR_BAD_OFFSETS: return "grouped offsets are not 0..T_total and non-decreasing";
        case I8QL_ERR_NO_DEVICE: return "no usable sm_103 CUDA device";
        case I8QL_ERR_WORKSPACE_LIMIT:
            return "workspace too small (w8a8_gemm_noalloc: M * K > 16 Mi for M > 32 exceeds its fixed array; "
                   "kv_cache_attention, kv_cache_weights: less than their workspace queries report)";
        case I8QL_ERR_BAD_INDEX: return "a cache slot, page, length, query offset or position is out of range";
        default: return "unknown status";
    }
}

int32_t i8ql_version(void) { return 1 * 10000 + 1 * 100 + 0; }

void i8ql_debug_stream_k_timeout(int32_t on) { g_debug_sk_timeout.store(on != 0 ? 1 : 0, std::memory_order_relaxed); }

void i8ql_set_early_weight_loads(int32_t on) { g_early_weights.store(on != 0 ? 1 : 0, std::memory_order_relaxed); }

int32_t i8ql_early_weight_loads(void) { return g_early_weights.load(std::memory_order_relaxed); }

}  // extern "C"

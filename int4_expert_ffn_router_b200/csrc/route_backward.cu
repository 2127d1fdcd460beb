// route_backward.cu -- gradient of the router's weights, rows and input
// (coli_moe_route_backward).
#include "block.cuh"

#define COLI_API extern "C" __attribute__((visibility("default")))

namespace coli {
namespace {

// dlogits[t][k] = w_k (dw_k - sum_j w_j dw_j): the weights are a softmax over
// the selected logits, whose Jacobian is diag(w) - w w^T. One warp a token.
__global__ void __launch_bounds__(256) route_dlogits_kernel(const int32_t* ids, const float* w, const float* dw, int T,
                                                            int K, int E, float* dl) {
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    float wk = 0.0f, gk = 0.0f;
    if (lane < K) {
        const size_t i = (size_t)t * K + lane;
        const int e = ids[i];
        wk = (unsigned)e < (unsigned)E ? w[i] : 0.0f;
        gk = wk != 0.0f ? dw[i] : 0.0f;  // an absent slot's dweights is not used
    }
    float m = wk * gk;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (lane < K) dl[(size_t)t * K + lane] = wk != 0.0f ? wk * (gk - m) : 0.0f;
}

// drouter_w[e] and dbias[e]: one block per expert and column tile walks the
// expert's slots in order.
template <typename XT, int V>
__global__ void __launch_bounds__(128) route_rows_kernel(const int32_t* offsets, const int32_t* slot, const float* dl,
                                                         int n, int K, const XT* x, int64_t ldx, int H, float* dwr,
                                                         float* dbias) {
    const int e = blockIdx.x;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int q0 = min(max(offsets[e], 0), n), q1 = min(offsets[e + 1], n);
    float acc[V], b = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int q = q0; q < q1; ++q) {
        const int i = slot[q];
        if (i < 0 || i >= n) continue;
        const float d = dl[i];
        if (d == 0.0f) continue;  // an absent slot: its token adds nothing, whatever it holds
        b += d;
        if (dwr && c < H) {
            Raw<XT, V> r;
            r.load(x + (size_t)(i / K) * ldx + c);
            float v[V];
            r.get(v);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = fmaf(d, v[j], acc[j]);
        }
    }
    if (dwr && c < H) {
        Raw<float, V> out;
        out.set(acc);
        out.store(dwr + (size_t)e * H + c);
    }
    if (dbias && blockIdx.y == 0 && threadIdx.x == 0) dbias[e] = b;
}

template <typename XT>
cudaError_t route_rows(const int32_t* offsets, const int32_t* slot, const float* dl, int T, int K, int E, const Mat& x,
                       float* dwr, float* dbias, cudaStream_t st) {
    const bool vec = x.cols % 8 == 0 && x.vec() && ((uintptr_t)dwr & 15u) == 0;
    const int V = vec ? 8 : 1;
    return launch(vec ? route_rows_kernel<XT, 8> : route_rows_kernel<XT, 1>,
                  dim3(E, dwr ? (x.cols + 128 * V - 1) / (128 * V) : 1), 128, 0, st, false, offsets, slot, dl, T * K, K,
                  (const XT*)x.p, x.stride, x.cols, dwr, dbias);
}

#define REQUIRE(cond, msg)                                \
    do {                                                  \
        if (!(cond)) return block_fail(COLI_EINVAL, msg); \
    } while (0)

}  // namespace
}  // namespace coli

using namespace coli;

COLI_API int64_t coli_moe_route_backward_workspace(int T, int K, int E, int H) {
    if (T < 0 || T > kBlockMaxTokens || K < 1 || K > 32 || (int64_t)T * K > kBlockMaxSlots || E < 1 || E > 1024 || H < 1 ||
        H > kBlockMaxHidden)
        return -1;
    return 0;
}

COLI_API coli_status coli_moe_route_backward(const float* router_w, int E, int H, int K, const void* x, coli_dtype dtype,
                                             int64_t x_stride, int T, const int32_t* ids, const float* weights,
                                             const float* dweights, const int32_t* offsets, const int32_t* slot,
                                             float* dlogits, void* dx, int64_t dx_stride, float* drouter_w,
                                             float* dbias, void* work, int64_t work_bytes, int device,
                                             coli_stream stream) {
    const int64_t need = coli_moe_route_backward_workspace(T, K, E, H);
    REQUIRE(need >= 0, "need 0 <= n_tokens <= 2^20, 1 <= top_k <= 32, n_tokens * top_k <= 2^24, 1 <= n_experts <= 1024, "
                       "1 <= hidden <= 65536");
    REQUIRE(dtype_ok(dtype), "dtype must be COLI_F32 or COLI_BF16");
    REQUIRE(device >= 0, "no such CUDA device");
    REQUIRE(need == 0 || (work && work_bytes >= need), "work is smaller than coli_moe_route_backward_workspace");
    REQUIRE(((uintptr_t)work & 15u) == 0, "work must be 16-byte aligned");
    const bool rows = drouter_w || dbias;
    const size_t n = (size_t)T * K * 4, wb = (size_t)E * H * 4;
    const Mat mx{x, dtype, T, H, x_stride}, mdx{dx, dtype, T, H, dx_stride}, mw{router_w, COLI_F32, E, H, H};
    if (T > 0) {
        REQUIRE(ids && weights && dweights && dlogits, "ids, weights, dweights or dlogits is NULL");
        if (drouter_w)
            if (const char* m = check_mat(mx, "x is NULL", "x_stride is smaller than hidden", "x is not aligned to its element"))
                return block_fail(COLI_EINVAL, m);
        if (dx) {
            if (const char* m = check_mat(mdx, "", "dx_stride is smaller than hidden", "dx is not aligned to its element"))
                return block_fail(COLI_EINVAL, m);
            REQUIRE(router_w, "router_w is NULL");
        }
        REQUIRE(!rows || (offsets && slot), "drouter_w and dbias need offsets and slot");
    }
    REQUIRE((((uintptr_t)router_w | (uintptr_t)ids | (uintptr_t)weights | (uintptr_t)dweights | (uintptr_t)offsets |
              (uintptr_t)slot | (uintptr_t)dlogits | (uintptr_t)drouter_w | (uintptr_t)dbias) & 3u) == 0,
            "int32 and fp32 arrays must be 4-byte aligned");
    const void* ins[] = {router_w, ids, weights, dweights, offsets, slot, drouter_w ? x : nullptr};
    const size_t il[] = {wb, n, n, n, (size_t)(E + 1) * 4, n, mx.bytes()};
    const void* outs[] = {dlogits, dx, drouter_w, dbias, need ? work : nullptr};
    const size_t ol[] = {n, dx ? mdx.bytes() : 0, wb, (size_t)E * 4, (size_t)need};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 6; ++j) REQUIRE(!overlap(outs[i], ol[i], ins[j], il[j]), "an output overlaps an input");
        if (drouter_w) REQUIRE(i == 1 ? !(dx && overlap(mdx, mx)) : !overlap(outs[i], ol[i], x, mx.bytes()), "an output overlaps x");
        for (int j = 0; j < i; ++j) REQUIRE(!overlap(outs[i], ol[i], outs[j], ol[j]), "two outputs overlap");
    }
    DeviceGuard guard(device);
    REQUIRE(guard.ok, "no such CUDA device");
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (T == 0) {  // sums over no tokens
        if (drouter_w) e = cudaMemsetAsync(drouter_w, 0, wb, st);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)E * 4, st);
        return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "route backward: clear");
    }
    e = launch(route_dlogits_kernel, (T + 7) / 8, 256, 0, st, false, ids, weights, dweights, T, K, E, dlogits);
    if (e != cudaSuccess) return block_cuda_fail(e, "route backward: logits");
    if (dx) {
        e = launch_gather_sum(ids, dlogits, T, K, mw, nullptr, mdx, st, false);
        if (e != cudaSuccess) return block_cuda_fail(e, "route backward: dx");
    }
    if (rows) {
        e = dtype == COLI_F32 ? route_rows<float>(offsets, slot, dlogits, T, K, E, mx, drouter_w, dbias, st)
                              : route_rows<__nv_bfloat16>(offsets, slot, dlogits, T, K, E, mx, drouter_w, dbias, st);
        if (e != cudaSuccess) return block_cuda_fail(e, "route backward: rows");
    }
    return COLI_OK;
}

// route_backward.cu -- gradient of the router's weights, rows and input
// (coli_moe_route_backward).
#include "block.cuh"

#define COLI_API extern "C" __attribute__((visibility("default")))

namespace coli {
namespace {

constexpr int kSms = 148;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// dlogits[t][k] = w_k (dw_k - sum_j w_j dw_j): the weights are a softmax over
// the selected logits, whose Jacobian is diag(w) - w w^T. One warp a token.
__global__ void __launch_bounds__(256) route_dlogits_kernel(const int32_t* ids, const float* w, const float* dw, int T,
                                                            int K, int E, float* dl) {
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t < T) {
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
    grid_next();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---------------------------------------------------------------------------
// dx[t] = sum_k dlogits[t][k] Wr[ids[t][k]]. Every token reads K router rows:
// at 2048 x 8 x 6144 that is 403 MB, against 6 MB of router. So a block keeps a
// slab of 32 * VC columns of all E rows in shared memory and takes a share of
// the tokens, one warp each, a lane VC columns: bound by shared memory reads
// (13 us at those sizes). A slot that is absent reads a row of zeros.
// ---------------------------------------------------------------------------
template <typename XT, int VC>
__global__ void __launch_bounds__(kThreads) route_dx_kernel(const int32_t* ids, const float* dl, const float* wr, int T,
                                                            int K, int E, int H, int per, bool vec, XT* dx, int64_t ldx) {
    extern __shared__ __align__(16) float slab[];  // [E + 1][32 * VC], the last row zero
    constexpr int C = 32 * VC;
    const int c0 = blockIdx.x * C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (vec) {
        for (int i = threadIdx.x; i < E * (C / 4); i += kThreads) {
            const int e = i / (C / 4), c = (i % (C / 4)) * 4;
            if (c0 + c < H) cp_async16(smem_addr(slab + e * C + c), wr + (size_t)e * H + c0 + c);
        }
    } else {
        for (int i = threadIdx.x; i < E * C; i += kThreads) {
            const int e = i / C, c = i % C;
            if (c0 + c < H) slab[i] = wr[(size_t)e * H + c0 + c];
        }
    }
    for (int i = threadIdx.x; i < C; i += kThreads) slab[E * C + i] = 0.0f;
    grid_wait();  // dlogits
    const int t1 = min(T, (int)(blockIdx.y + 1) * per);
    int t = blockIdx.y * per + warp;
    auto fetch = [&](int at, int& e, float& d) {
        e = E;
        d = 0.0f;
        if (at < t1 && lane < K) {
            d = dl[(size_t)at * K + lane];
            const int id = ids[(size_t)at * K + lane];
            e = d != 0.0f && (unsigned)id < (unsigned)E ? id : E;
        }
    };
    int e;
    float d;
    fetch(t, e, d);
    cp_async_wait_all();
    __syncthreads();
    const float* mine = slab + lane * VC;
    const int left = H - c0 - lane * VC;
    for (; t < t1; t += kWarps) {
        int e1;
        float d1;
        fetch(t + kWarps, e1, d1);
        float acc[VC];
#pragma unroll
        for (int j = 0; j < VC; ++j) acc[j] = 0.0f;
        for (int k0 = 0; k0 < K; k0 += 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // lanes from K on hold the zero row
                const int ek = __shfl_sync(0xffffffffu, e, k0 + k);
                const float dk = __shfl_sync(0xffffffffu, d, k0 + k);
                const float* row = mine + ek * C;
                if constexpr (VC == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(row);
                    acc[0] = fmaf(dk, v.x, acc[0]);
                    acc[1] = fmaf(dk, v.y, acc[1]);
                    acc[2] = fmaf(dk, v.z, acc[2]);
                    acc[3] = fmaf(dk, v.w, acc[3]);
                } else if constexpr (VC == 2) {
                    const float2 v = *reinterpret_cast<const float2*>(row);
                    acc[0] = fmaf(dk, v.x, acc[0]);
                    acc[1] = fmaf(dk, v.y, acc[1]);
                } else {
                    acc[0] = fmaf(dk, row[0], acc[0]);
                }
            }
        }
        XT* out = dx + (size_t)t * ldx + c0 + lane * VC;
        if (VC == 4 && vec) {
            if (left > 0) {
                if constexpr (sizeof(XT) == 4) {
                    *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1 % VC], acc[2 % VC], acc[3 % VC]);
                } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0], acc[1 % VC]), hi = __floats2bfloat162_rn(acc[2 % VC], acc[3 % VC]);
                    *reinterpret_cast<uint2*>(out) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VC; ++j)
                if (j < left) {
                    Raw<XT, 1> r;
                    const float one[1] = {acc[j]};
                    r.set(one);
                    r.store(out + j);
                }
        }
        e = e1;
        d = d1;
    }
    grid_next();
}

// ---------------------------------------------------------------------------
// drouter_w[e] and dbias[e]: sums over the expert's slots of dlogits * x[token].
// Again a token's row is needed K times, so a block keeps 256 bytes of columns
// of up to kChunk tokens in shared memory; a warp takes an expert and adds the
// chunk's slots of that expert (found in its sorted list by bisection) in
// order, two rows at a time, sixteen lanes each. A block's sums go to its
// split's part of the workspace, which route_sum_kernel adds in order; with one
// split they are the result. At 2048 x 8 x 6144 bf16: 25 MB of x once, bound by
// the instructions that widen and add the 201 MB of rows.
// ---------------------------------------------------------------------------
constexpr int kRowBytes = 256;
constexpr int kChunk = 704;

// First index in [a, b) whose slot is >= bound (the list of an expert is ascending).
__device__ __forceinline__ int first_at_least(const int32_t* slot, int a, int b, int bound) {
    while (a < b) {
        const int m = (a + b) >> 1;
        if (slot[m] < bound) a = m + 1;
        else b = m;
    }
    return a;
}

template <typename XT>
__global__ void __launch_bounds__(kThreads) route_rows_kernel(const int32_t* offsets, const int32_t* slot, const float* dl,
                                                              int T, int K, int E, const XT* x, int64_t ldx, int H, int per,
                                                              bool vec, bool vec_out, float* part, float* part_b) {
    extern __shared__ __align__(16) unsigned char rows[];  // [kChunk + 1][256], the last row zero; then int [2][E]
    __shared__ int next;
    constexpr int C = kRowBytes / sizeof(XT), V = 16 / sizeof(XT);
    int* cur = reinterpret_cast<int*>(rows + (kChunk + 1) * kRowBytes);
    int* end = cur + E;
    const int c0 = blockIdx.x * C, lane = threadIdx.x & 31, half = lane >> 4, at = lane & 15;
    const int n = T * K, ta = blockIdx.y * per, tb = min(T, ta + per);
    for (int e = threadIdx.x; e < E; e += kThreads) {
        const int q0 = min(max(offsets[e], 0), n), q1 = min(max(offsets[e + 1], q0), n);
        cur[e] = first_at_least(slot, q0, q1, ta * K);
    }
    if (threadIdx.x < kRowBytes / 4) reinterpret_cast<int*>(rows + kChunk * kRowBytes)[threadIdx.x] = 0;
    for (int t0 = ta; t0 < tb || t0 == ta; t0 += kChunk) {
        const int t1 = min(tb, t0 + kChunk);
        if (part) {
            if (vec) {
                for (int i = threadIdx.x; i < (t1 - t0) * 16; i += kThreads) {
                    const int t = i >> 4, c = (i & 15) * V;
                    if (c0 + c < H) cp_async16(smem_addr(rows) + i * 16, x + (size_t)(t0 + t) * ldx + c0 + c);
                }
            } else {
                for (int i = threadIdx.x; i < (t1 - t0) * C; i += kThreads) {
                    const int t = i / C, c = i % C;
                    if (c0 + c < H) reinterpret_cast<XT*>(rows)[i] = x[(size_t)(t0 + t) * ldx + c0 + c];
                }
            }
        }
        for (int e = threadIdx.x; e < E; e += kThreads) {
            const int q1 = min(max(offsets[e + 1], 0), n);
            end[e] = first_at_least(slot, cur[e], max(q1, cur[e]), t1 * K);
        }
        if (threadIdx.x == 0) next = 0;
        if (t0 == ta) grid_wait();  // dlogits
        cp_async_wait_all();
        __syncthreads();
        for (;;) {
            int e = 0;
            if (lane == 0) e = atomicAdd(&next, 1);  // which warp takes an expert does not show in its sum
            e = __shfl_sync(0xffffffffu, e, 0);
            if (e >= E) break;
            const int q1 = end[e];
            float acc[V], b = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = 0.0f;
            for (int q = cur[e]; q < q1; q += 32) {
                int r = kChunk;  // the zero row: an absent slot, or one that is not of this chunk
                float d = 0.0f;
                if (q + lane < q1) {
                    const int i = slot[q + lane];
                    if (i >= t0 * K && i < t1 * K) {
                        d = dl[i];
                        if (d != 0.0f) r = i / K - t0;
                    }
                }
                b += d;
                if (!part) continue;
                const int steps = (min(32, q1 - q) + 1) >> 1;
                for (int s0 = 0; s0 < steps; s0 += 4) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {  // steps behind the last take the zero row
                        const int src = 2 * (s0 + s) + half;
                        const int rr = __shfl_sync(0xffffffffu, r, src);
                        const float dd = __shfl_sync(0xffffffffu, d, src);
                        const uint4 u = *reinterpret_cast<const uint4*>(rows + rr * kRowBytes + at * 16);
                        if constexpr (sizeof(XT) == 4) {
                            acc[0] = fmaf(dd, __uint_as_float(u.x), acc[0]);
                            acc[1] = fmaf(dd, __uint_as_float(u.y), acc[1]);
                            acc[2] = fmaf(dd, __uint_as_float(u.z), acc[2]);
                            acc[3] = fmaf(dd, __uint_as_float(u.w), acc[3]);
                        } else {
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                acc[(2 * j) % V] = fmaf(dd, __uint_as_float(w[j] << 16), acc[(2 * j) % V]);
                                acc[(2 * j + 1) % V] = fmaf(dd, __uint_as_float(w[j] & 0xffff0000u), acc[(2 * j + 1) % V]);
                            }
                        }
                    }
                }
            }
            if (part) {
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 16);
                const int c = c0 + at * V;
                float* out = part + ((size_t)blockIdx.y * E + e) * H + c;
                if (half == 0 && c < H) {
                    if (vec_out) {
#pragma unroll
                        for (int j = 0; j < V; j += 4) {
                            float4 v = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                            if (t0 != ta) {
                                const float4 o = *reinterpret_cast<const float4*>(out + j);
                                v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
                            }
                            *reinterpret_cast<float4*>(out + j) = v;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (c + j < H) out[j] = t0 != ta ? out[j] + acc[j] : acc[j];
                    }
                }
            }
            if (part_b && blockIdx.x == 0) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
                float* out = part_b + (size_t)blockIdx.y * E + e;
                if (lane == 0) *out = t0 != ta ? *out + b : b;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kThreads) cur[e] = end[e];
    }
    grid_next();
}

// out[i] = sum over the splits of part[s][i], in order; V values a thread.
template <int V>
__global__ void __launch_bounds__(256) route_sum_kernel(const float* part, int splits, int n, float* dwr,
                                                        const float* part_b, int E, float* dbias) {
    grid_wait();
    const int i = (blockIdx.x * 256 + threadIdx.x) * V;
    if (dwr && i < n) {
        float acc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float* p = part + (size_t)s * n + i;
            if constexpr (V == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
                acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
            } else {
                acc[0] += __ldcg(p);
            }
        }
        if constexpr (V == 4) *reinterpret_cast<float4*>(dwr + i) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else dwr[i] = acc[0];
    }
    if (dbias && blockIdx.x * 256 + threadIdx.x < E) {
        float b = 0.0f;
        for (int s = 0; s < splits; ++s) b += __ldcg(part_b + (size_t)s * E + blockIdx.x * 256 + threadIdx.x);
        dbias[blockIdx.x * 256 + threadIdx.x] = b;
    }
}

// Splits of the tokens: as many as fill the GPU beside the column slabs, each
// of 128 tokens or more (the workspace's size depends on it; it must not
// depend on the type: the fewer slabs, of bf16, count).
struct Split {
    int n, per;
};
Split split_of(int T, int H) {
    const int slabs = (H + 127) / 128;
    int n = kSms / slabs;
    if (n > (T + 127) / 128) n = (T + 127) / 128;
    if (n < 1) n = 1;
    const int per = T > 0 ? (T + n - 1) / n : 1;
    return {T > 0 ? (T + per - 1) / per : 1, per};
}

template <typename XT>
cudaError_t route_rows(const int32_t* offsets, const int32_t* slot, const float* dl, int T, int K, int E, const Mat& x,
                       float* dwr, float* dbias, void* work, cudaStream_t st) {
    constexpr int C = kRowBytes / sizeof(XT);
    const int H = x.cols;
    const Split sp = split_of(T, H);
    const bool vec = x.vec() && H % (16 / sizeof(XT)) == 0;
    // one split writes the result itself, several their parts
    float* part = sp.n > 1 ? (float*)work : dwr;
    float* part_b = sp.n > 1 ? (float*)work + (size_t)sp.n * E * H : dbias;
    const bool vec_out = H % 4 == 0 && ((uintptr_t)part & 15u) == 0 && H % (16 / sizeof(XT)) == 0;
    const size_t smem = (size_t)(kChunk + 1) * kRowBytes + (size_t)2 * E * 4;
    cudaError_t e = cudaFuncSetAttribute(route_rows_kernel<XT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch(route_rows_kernel<XT>, dim3(dwr ? (H + C - 1) / C : 1, sp.n), kThreads, smem, st, true, offsets, slot, dl, T, K,
               E, (const XT*)x.p, x.stride, H, sp.per, vec, vec_out, dwr ? part : nullptr, dbias ? part_b : nullptr);
    if (e != cudaSuccess || sp.n == 1) return e;
    const int n = E * H;
    const bool v4 = H % 4 == 0 && (((uintptr_t)dwr | (uintptr_t)work) & 15u) == 0;
    const int V = v4 ? 4 : 1, blocks = dwr ? (n / V + 255) / 256 : 1, need = (E + 255) / 256;
    return launch(v4 ? route_sum_kernel<4> : route_sum_kernel<1>, blocks > need ? blocks : need, 256, 0, st, true,
                  (const float*)part, sp.n, n, dwr, (const float*)part_b, E, dbias);
}

// Columns of a slab of all E router rows (and the zero row) in shared memory.
int slab_columns(int E) {
    for (int vc : {4, 2}) if ((size_t)(E + 1) * 32 * vc * 4 <= 200 * 1024) return vc;
    return 1;
}

template <typename XT>
cudaError_t route_dx(const int32_t* ids, const float* dl, const Mat& wr, int T, int K, const Mat& dx, cudaStream_t st) {
    const int E = (int)wr.rows, H = wr.cols, vc = slab_columns(E), C = 32 * vc;
    const int slabs = (H + C - 1) / C;
    int n = kSms / slabs;
    if (n > (T + kWarps - 1) / kWarps) n = (T + kWarps - 1) / kWarps;
    if (n < 1) n = 1;
    const int per = (T + n - 1) / n;
    const bool vec = H % 4 == 0 && wr.vec() && dx.vec();
    const size_t smem = (size_t)(E + 1) * C * 4;
    auto k = vc == 4 ? route_dx_kernel<XT, 4> : vc == 2 ? route_dx_kernel<XT, 2> : route_dx_kernel<XT, 1>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch(k, dim3(slabs, (T + per - 1) / per), kThreads, smem, st, true, ids, dl, (const float*)wr.p, T, K, E, H, per,
                  vec, (XT*)dx.p, dx.stride);
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
    const int n = split_of(T, H).n;
    return n > 1 ? (int64_t)n * E * ((int64_t)H + 1) * 4 : 0;
}

COLI_API coli_status coli_moe_route_backward(const float* router_w, int E, int H, int K, const void* x, coli_dtype dtype,
                                             int64_t x_stride, int T, const int32_t* ids, const float* weights,
                                             const float* dweights, const int32_t* offsets, const int32_t* slot,
                                             float* dlogits, void* dx, int64_t dx_stride, float* drouter_w,
                                             float* dbias, void* work, int64_t work_bytes, int device,
                                             coli_stream stream) {
    const bool rows = drouter_w || dbias;
    const int64_t size = coli_moe_route_backward_workspace(T, K, E, H);
    REQUIRE(size >= 0, "need 0 <= n_tokens <= 2^20, 1 <= top_k <= 32, n_tokens * top_k <= 2^24, 1 <= n_experts <= 1024, "
                       "1 <= hidden <= 65536");
    const int64_t need = rows && T > 0 ? size : 0;
    REQUIRE(dtype_ok(dtype), "dtype must be COLI_F32 or COLI_BF16");
    REQUIRE(device >= 0, "no such CUDA device");
    REQUIRE(need == 0 || (work && work_bytes >= need), "work is smaller than coli_moe_route_backward_workspace");
    REQUIRE(((uintptr_t)work & 15u) == 0, "work must be 16-byte aligned");
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
    const void* ins[] = {router_w, ids, weights, dweights, offsets, slot};
    const size_t il[] = {wb, n, n, n, (size_t)(E + 1) * 4, n};
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
        // few slots read fewer router rows than a slab of all of them holds
        if ((int64_t)T * K < E) e = launch_gather_sum(ids, dlogits, T, K, mw, nullptr, mdx, st, true);
        else e = dtype == COLI_F32 ? route_dx<float>(ids, dlogits, mw, T, K, mdx, st)
                                   : route_dx<__nv_bfloat16>(ids, dlogits, mw, T, K, mdx, st);
        if (e != cudaSuccess) return block_cuda_fail(e, "route backward: dx");
    }
    if (rows) {
        e = dtype == COLI_F32 ? route_rows<float>(offsets, slot, dlogits, T, K, E, mx, drouter_w, dbias, work, st)
                              : route_rows<__nv_bfloat16>(offsets, slot, dlogits, T, K, E, mx, drouter_w, dbias, work, st);
        if (e != cudaSuccess) return block_cuda_fail(e, "route backward: rows");
    }
    return COLI_OK;
}

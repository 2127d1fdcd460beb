// block.cuh -- shared parts of the operators around an MoE block (dispatch.cu,
// block_norm.cu, route_backward.cu): row access, reductions, launches, checks.
#pragma once

#include <string>

#include "common.cuh"
#include "kernels.cuh"

namespace coli {

// Switches to `dev` for the lifetime of the guard.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
        if (!ok) cudaGetLastError();  // reported by the caller, not left behind
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// Records a failure of an operator's C entry (no exception leaves it).
inline coli_status block_fail(coli_status s, const char* what) {
    try {
        set_last_error(what);
    } catch (...) {
    }
    return s;
}
inline coli_status block_cuda_fail(cudaError_t e, const char* where) {
    try {
        set_last_error(std::string(where) + ": " + cudaGetErrorString(e));
    } catch (...) {
    }
    return COLI_ECUDA;
}

constexpr int kBlockMaxHidden = 65536;
constexpr int kBlockMaxTokens = 1 << 20;
constexpr int64_t kBlockMaxSlots = 1 << 24;

inline bool dtype_ok(coli_dtype t) { return t == COLI_F32 || t == COLI_BF16; }
inline size_t dtype_size(coli_dtype t) { return t == COLI_F32 ? 4 : 2; }

// A row-major matrix argument: rows of `cols` values, `stride` values apart.
struct Mat {
    const void* p;
    coli_dtype t;
    int64_t rows;
    int cols;
    int64_t stride;
    // bytes from the first value to the end of the last
    size_t bytes() const { return rows > 0 ? ((size_t)(rows - 1) * stride + cols) * dtype_size(t) : 0; }
    bool aligned(size_t n) const { return ((uintptr_t)p % n) == 0; }
    // rows start on n-byte boundaries (one row: its start alone)
    bool starts(size_t n) const { return aligned(n) && (rows <= 1 || (size_t)stride * dtype_size(t) % n == 0); }
    // V values a thread can be read and written at a time, by accesses of up to 16 bytes
    bool takes(int V) const {
        const size_t n = V * dtype_size(t);
        return cols % V == 0 && starts(n < 16 ? n : 16);
    }
};

inline const char* check_mat(const Mat& m, const char* null_msg, const char* stride_msg, const char* align_msg) {
    if (m.rows == 0) return nullptr;
    if (!m.p) return null_msg;
    if (m.stride < m.cols) return stride_msg;
    if (m.stride > ((int64_t)1 << 40)) return stride_msg;
    if (!m.aligned(dtype_size(m.t))) return align_msg;
    return nullptr;
}

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uint8_t *x = (const uint8_t*)a, *y = (const uint8_t*)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}
inline bool overlap(const Mat& a, const Mat& b) {
    if (!overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
    const int64_t s = a.stride * (int64_t)dtype_size(a.t);
    if (a.rows > 1 && b.rows > 1 && s == b.stride * (int64_t)dtype_size(b.t)) {  // columns of one wider matrix
        const int64_t d = (((int64_t)((uintptr_t)b.p - (uintptr_t)a.p)) % s + s) % s;
        return d < a.cols * (int64_t)dtype_size(a.t) || s - d < b.cols * (int64_t)dtype_size(b.t);
    }
    return true;
}
// The same matrix (an operator that reads each value before it writes it takes this).
inline bool same(const Mat& a, const Mat& b) { return a.p == b.p && a.t == b.t && a.stride == b.stride; }

// Launches `kernel`, in clusters of `cluster` blocks. dependent: it may start
// while the kernel before it on the stream still runs, and waits for that one's
// results itself (grid_wait).
template <typename... P, typename... A>
cudaError_t launch_clusters(int cluster, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            bool dependent, A... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[2];
    c.attrs = at;
    if (dependent) {
        at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[c.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[c.numAttrs].val.clusterDim.x = cluster;
        at[c.numAttrs].val.clusterDim.y = 1;
        at[c.numAttrs++].val.clusterDim.z = 1;
    }
    return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool dependent, A... args) {
    return launch_clusters(1, kernel, grid, block, smem, st, dependent, args...);
}
// Lets `kernel` take dynamic shared memory of up to `most` bytes. The limit is one
// for all callers of a kernel on a device, so it is the most that any call
// takes: of two threads' calls one would otherwise lower it under the other's launch.
template <typename... P>
cudaError_t allow_shared(void (*kernel)(P...), size_t most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}
// Waits until the kernels before this one have finished and their writes can be read.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream start (its grid_wait still waits for this one's end).
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------
// V consecutive values of a row as fp32: 8, 4, 2 or 1, by accesses of up to 16
// bytes (Mat::takes). The loads are volatile asm, so an in-place operator's loads and
// stores keep their order.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ void st16(void* p, uint4 r) {
    asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w) : "memory");
}

// The bits of V values, as loaded.
template <typename T, int V>
struct Raw;
template <>
struct Raw<float, 8> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) { a = ld16(p); b = ld16(p + 4); }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    }
    __device__ __forceinline__ void store(float* p) const { st16(p, a); st16(p + 4, b); }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld16(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);  // nearest, ties to even
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        a = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { st16(p, a); }
};
// Four or two values: rows whose starts allow 16, 8 or 4 bytes at a time.
template <>
struct Raw<float, 4> {
    uint4 a;
    __device__ __forceinline__ void load(const float* p) { a = ld16(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    }
    __device__ __forceinline__ void set(const float (&v)[4]) {
        a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    __device__ __forceinline__ void store(float* p) const { st16(p, a); }
};
template <>
struct Raw<float, 2> {
    uint2 a;
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(a.x), "=r"(a.y) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { a = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&v)[2]) const { v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); }
    __device__ __forceinline__ void set(const float (&v)[2]) { a = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1])); }
    __device__ __forceinline__ void store(float* p) const { asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(a.x), "r"(a.y) : "memory"); }
};
template <>
struct Raw<__nv_bfloat16, 4> {
    uint2 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(a.x), "=r"(a.y) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { a = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
        v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
    }
    __device__ __forceinline__ void set(const float (&v)[4]) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]), l = __floats2bfloat162_rn(v[2], v[3]);
        a = make_uint2(*reinterpret_cast<const uint32_t*>(&h), *reinterpret_cast<const uint32_t*>(&l));
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const {
        asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(a.x), "r"(a.y) : "memory");
    }
};
template <>
struct Raw<__nv_bfloat16, 2> {
    uint32_t a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { asm volatile("ld.global.u32 %0, [%1];" : "=r"(a) : "l"(p) : "memory"); }
    __device__ __forceinline__ void zero() { a = 0; }
    __device__ __forceinline__ void get(float (&v)[2]) const { v[0] = __uint_as_float(a << 16); v[1] = __uint_as_float(a & 0xffff0000u); }
    __device__ __forceinline__ void set(const float (&v)[2]) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
        a = *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { asm volatile("st.global.u32 [%0], %1;" ::"l"(p), "r"(a) : "memory"); }
};
template <>
struct Raw<float, 1> {
    float a;
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(a) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { a = 0.0f; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = a; }
    __device__ __forceinline__ void set(const float (&v)[1]) { a = v[0]; }
    __device__ __forceinline__ void store(float* p) const { asm volatile("st.global.f32 [%0], %1;" ::"l"(p), "f"(a) : "memory"); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    unsigned short a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(a) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { a = 0; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __uint_as_float((uint32_t)a << 16); }
    __device__ __forceinline__ void set(const float (&v)[1]) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v[0]);
        a = *reinterpret_cast<const unsigned short*>(&h);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { asm volatile("st.global.u16 [%0], %1;" ::"l"(p), "h"(a) : "memory"); }
};

// Sums of NR values over the block, in every thread, in a fixed order. `red`
// holds 32 * NR values; consecutive calls must alternate between two of them
// (one barrier a call: a warp may still read the buffer of the call before).
template <typename F, int NR>
__device__ __forceinline__ void block_sum(F (&v)[NR], F* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < NR; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    if (lane == 0)
#pragma unroll
        for (int r = 0; r < NR; ++r) red[warp * NR + r] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NR; ++r) v[r] = lane < nw ? red[lane * NR + r] : F(0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < NR; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
}

// dispatch.cu: y[t] = base[t] + sum_k w[t][k] rows[pos[t][k]] over the positions in
// [0, rows.rows) (w NULL: 1; skip_zero: a slot of weight 0 is left out, whatever
// its row holds). y, base: [T][H] of one type; dependent: see launch().
cudaError_t launch_gather_sum(const int32_t* pos, const float* w, bool skip_zero, int T, int K, const Mat& rows,
                              const Mat* base, const Mat& y, cudaStream_t st, bool dependent);

// block_norm.cu: the norms around a block (coli_block_norm), arguments checked by the caller.
coli_status block_norm_launch(const coli_block_params* prev, const coli_block_params* next, const Mat* x, const Mat* y,
                              const Mat* x_out, const Mat* n, const float* token_gate, int T, int H, cudaStream_t st);
const char* check_block_params(const coli_block_params* p);

}  // namespace coli

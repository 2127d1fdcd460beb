// block_norm.cu -- the norms around a block with its gate and scales
// (coli_block_norm) and their gradients.
#include "block.cuh"

#include <initializer_list>

#define COLI_API extern "C" __attribute__((visibility("default")))

namespace coli {
namespace {

struct NormArgs {
    int T, H;
    const void *x, *y;      // forward: x; backward: x_out (s)
    int64_t ldx, ldy;
    const float *pre, *post, *gate, *token;  // gains, channel gate, token gate (NULL: 1)
    float xs, ys, eps_post, eps_pre;
    int has_prev, has_next, post_norm;
    // forward
    void *xo, *n;
    int64_t ldxo, ldn;
    // backward
    const void *dxo, *dn;
    int64_t lddxo, lddn;
    void *dx, *dy;
    int64_t lddx, lddy;
    float *dtoken;
    float* part;            // [grid][2][H] the blocks' sums over their rows of s r dn and of u y rho ds (NULL: not wanted)
    int stages;             // slots of the ring in shared memory (0: none)
};

// A sum of squares that fp32 holds well: it neither overflowed nor lost to
// underflow anything that eps does not hide (a square below 2^-126 is lost).
__device__ __forceinline__ bool sum_ok(float ss, float eps) { return ss <= 3e37f && (ss >= 1e-24f || eps >= 1e-12f); }
__device__ __forceinline__ float rms_scale(double ss, int H, float eps) { return (float)(1.0 / sqrt(ss / H + (double)eps)); }

// A column's gain or gate (NULL: 1).
__device__ __forceinline__ float gain(const float* g, int c) { return g ? __ldg(g + c) : 1.0f; }

// ---------------------------------------------------------------------------
// A thread holds N pieces of V columns of a row: V = 8 where all rows are bf16,
// V = 4 where some are fp32 (so that a warp's 16-byte accesses lie side by side:
// two of them 32 bytes apart read every 32-byte sector twice, and took 1.6 times
// as long), both for rows whose starts allow it; else V = 2, read one by one.
// Arithmetic is on pairs of columns (fp32 x 2 instructions): a row's
// instructions, not its bytes, bound these kernels otherwise.
//
// A block takes the rows b, b + grid, ...: the columns' parameters are read
// once, and with V >= 4 the next rows are copied into a ring in shared memory
// (cp.async) while a row is worked on. A thread copies what it alone reads, so
// the ring needs no barrier.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 bf16_pair(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t to_bf16_pair(float2 v) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);  // nearest, ties to even
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint2 ld8(const void* p) {
    uint2 r;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
    return r;
}

template <typename T, int V>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        v[0] = bf16_pair(w.x); v[1] = bf16_pair(w.y); v[2] = bf16_pair(w.z); v[3] = bf16_pair(w.w);
    }
    __device__ __forceinline__ void set(const float2 (&v)[4]) {
        w = make_uint4(to_bf16_pair(v[0]), to_bf16_pair(v[1]), to_bf16_pair(v[2]), to_bf16_pair(v[3]));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int) { w = ld16(p); }
    __device__ __forceinline__ void load_shared(uint32_t at) { w = lds16(at); }
    __device__ __forceinline__ void store(__nv_bfloat16* p, int) const { st16(p, w); }
};
template <>
struct Piece<float, 4> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 (&v)[2]) const {
        v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    __device__ __forceinline__ void set(const float2 (&v)[2]) {
        w = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    }
    __device__ __forceinline__ void load(const float* p, int) { w = ld16(p); }
    __device__ __forceinline__ void load_shared(uint32_t at) { w = lds16(at); }
    __device__ __forceinline__ void store(float* p, int) const { st16(p, w); }
};
template <>
struct Piece<__nv_bfloat16, 4> {
    uint2 w;
    __device__ __forceinline__ void zero() { w = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float2 (&v)[2]) const { v[0] = bf16_pair(w.x); v[1] = bf16_pair(w.y); }
    __device__ __forceinline__ void set(const float2 (&v)[2]) { w = make_uint2(to_bf16_pair(v[0]), to_bf16_pair(v[1])); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int) { w = ld8(p); }
    __device__ __forceinline__ void load_shared(uint32_t at) { w = lds8(at); }
    __device__ __forceinline__ void store(__nv_bfloat16* p, int) const {
        asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(w.x), "r"(w.y) : "memory");
    }
};
// Two columns, the second of which may lie behind the row's end (left == 1).
template <typename T>
struct Piece<T, 2> {
    Raw<T, 1> a, b;
    __device__ __forceinline__ void zero() { a.zero(); b.zero(); }
    __device__ __forceinline__ void get(float2 (&v)[1]) const {
        float x[1], y[1];
        a.get(x);
        b.get(y);
        v[0] = make_float2(x[0], y[0]);
    }
    __device__ __forceinline__ void set(const float2 (&v)[1]) {
        const float x[1] = {v[0].x}, y[1] = {v[0].y};
        a.set(x);
        b.set(y);
    }
    __device__ __forceinline__ void load(const T* p, int left) {
        a.load(p);
        if (left > 1) b.load(p + 1);
        else b.zero();
    }
    __device__ __forceinline__ void store(T* p, int left) const {
        a.store(p);
        if (left > 1) b.store(p + 1);
    }
};

template <int bytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for the oldest of the groups in flight (stages - 1 of them, or one).
__device__ __forceinline__ void cp_async_wait(int stages) {
    if (stages >= 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A piece of every thread lies side by side in a ring slot.
template <typename T, int V>
constexpr int kBytes = V * (int)sizeof(T);
template <typename T, int V, int N>
__device__ __forceinline__ uint32_t ring_bytes() { return (uint32_t)(N * blockDim.x * kBytes<T, V>); }
template <typename T, int V>
__device__ __forceinline__ uint32_t ring_place(uint32_t array, int i) {
    return array + (i * blockDim.x + threadIdx.x) * kBytes<T, V>;
}

// Copies this thread's pieces of a row (row: its first column's address) to an array of a slot.
template <typename T, int V, int N>
__device__ __forceinline__ void ring_copy(uint32_t array, const T* row, int H) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if ((int)(i * blockDim.x + threadIdx.x) * V < H)
            cp_async<kBytes<T, V>>(ring_place<T, V>(array, i), row + i * blockDim.x * V);
}
// Zeroes this thread's places in the ring that no copy fills: columns behind
// the row's end, and (all) an array that is absent. Reads then need no conditions.
template <typename T, int V, int N>
__device__ __forceinline__ void ring_clear(uint32_t array, bool all, int H) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (all || (int)(i * blockDim.x + threadIdx.x) * V >= H) {
            const uint32_t at = ring_place<T, V>(array, i);
            if constexpr (kBytes<T, V> == 16) asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
            else asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(at), "r"(0) : "memory");
        }
}
// This thread's piece i of a row: from its ring slot, or from memory (row: its first column's address).
template <typename T, int V, bool ring>
__device__ __forceinline__ void take(Piece<T, V>& r, bool on, int i, uint32_t array, const T* row, int H) {
    if constexpr (ring) {
        r.load_shared(ring_place<T, V>(array, i));
    } else {
        const int left = H - (int)(i * blockDim.x + threadIdx.x) * V;
        r.zero();
        if (on && left > 0) r.load(row + i * blockDim.x * V, left);
    }
}

// Sums over the block (at most 16 warps) of NR values, 1 or 5 to 8, in every
// thread, in a fixed order. `red`: 16 * 8 floats, two of them in turn (one
// barrier a call).
__device__ __forceinline__ void block_sums(float (&v)[1], float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    if (lane == 0) red[warp] = v[0];
    __syncthreads();
    v[0] = lane < nw ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o >= 1; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    v[0] = __shfl_sync(0xffffffffu, v[0], 0);
}
// With every exchange a lane keeps half of its values (9 shuffles for 8
// values), then every warp adds the warps' sums, lane l those of value l % 8.
template <int NR>
__device__ __forceinline__ void block_sums(float (&v)[NR], float* red) {
    static_assert(NR > 4 && NR <= 8, "8 values a lane");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < NR ? v[j] : 0.0f;
#pragma unroll
    for (int half = 4; half >= 1; half /= 2) {
        const bool up = lane & (4 * half);
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const float keep = up ? w[j + half] : w[j], send = up ? w[j] : w[j + half];
            w[j] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * half);
        }
    }
    w[0] += __shfl_xor_sync(0xffffffffu, w[0], 2);
    w[0] += __shfl_xor_sync(0xffffffffu, w[0], 1);
    if ((lane & 3) == 0) red[warp * 8 + lane / 4] = w[0];
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        if (i + lane / 8 < nw) t += red[i * 8 + lane];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
#pragma unroll
    for (int j = 0; j < NR; ++j) v[j] = __shfl_sync(0xffffffffu, t, j);
}

// An array's columns c, c + 1, .. of a piece (NULL: 1); what lies behind the row's end is 0.
template <int V>
__device__ __forceinline__ void load_columns(const float* g, int c, int H, float2 (&v)[V / 2]) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) v[j] = both(c < H && !g ? 1.0f : 0.0f);
    if constexpr (V >= 4) {
        if (c >= H || !g) return;
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(g + c) + j);
            v[2 * j] = make_float2(f.x, f.y);
            v[2 * j + 1] = make_float2(f.z, f.w);
        }
    } else {
        if (g && c < H) v[0].x = __ldg(g + c);
        if (g && c + 1 < H) v[0].y = __ldg(g + c + 1);
        if (c + 1 >= H) v[0].y = 0.0f;
    }
}
// The branch's factor of each column: y_scale * gate * post_gain.
template <int V>
__device__ __forceinline__ void load_branch(const NormArgs& a, int c, float2 (&b)[V / 2]) {
    float2 p[V / 2];
    load_columns<V>(a.gate, c, a.H, b);
    load_columns<V>(a.post, c, a.H, p);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) b[j] = __fmul2_rn(b[j], __fmul2_rn(both(a.ys), p[j]));
}

// Sum of squares of a thread's pieces, in fp64 (rows beyond fp32's range).
template <typename T, int V, int N>
__device__ __forceinline__ double squares64(const Piece<T, V> (&r)[N]) {
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float2 v[V / 2];
        r[i].get(v);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) d += (double)v[j].x * v[j].x + (double)v[j].y * v[j].y;
    }
    return d;
}
// 1 / rms of a row held by the block.
template <typename T, int V, int N, bool wide>
__device__ __forceinline__ float row_scale(const Piece<T, V> (&r)[N], int H, float inv, float eps, float* red, double* red64) {
    float2 acc = both(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float2 v[V / 2];
        r[i].get(v);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) acc = __ffma2_rn(v[j], v[j], acc);
    }
    float ss[1] = {acc.x + acc.y};
    if constexpr (wide) block_sum<float, 1>(ss, red);  // up to 32 warps
    else block_sums(ss, red);
    if (__builtin_expect(sum_ok(ss[0], eps), 1)) return rsqrtf(fmaf(ss[0], inv, eps));
    double dd[1] = {squares64<T, V, N>(r)};
    block_sum<double, 1>(dd, red64);
    return rms_scale(dd[0], H, eps);
}

// The launch bound of 80 registers lets two blocks of 384 threads share an SM,
// one row's sums under the other's copies: 2048 x 6144 bf16 (101 MB) took 20 us,
// with one block an SM 23.
constexpr int kForwardThreads = 768;

// `single`: one row a block, read straight into registers by twice the threads.
// Such a launch is as long as its code, since it runs all of it once from cold
// instruction caches: with the ring one row of 6144 fp32 takes 5.4 us, without 4.2.
template <typename XT, typename YT, typename NT, int V, int N, bool single>
__global__ void __launch_bounds__(kForwardThreads) block_norm_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    __shared__ double red64[2][32];
    extern __shared__ __align__(16) unsigned char ring_mem[];
    const int H = a.H, stages = a.stages, c0 = threadIdx.x * V;
    const bool has_prev = a.has_prev, post = a.post_norm, has_next = a.has_next;
    const float inv = 1.0f / (float)H;
    constexpr bool kRing = V >= 4 && !single;
    const uint32_t xb = kRing ? ring_bytes<XT, V, N>() : 0;
    const uint32_t slot_bytes = kRing ? xb + ring_bytes<YT, V, N>() : 0;
    const uint32_t ring = smem_addr(ring_mem);
    if constexpr (kRing)
        for (int i = 0; i < stages; ++i) {
            ring_clear<XT, V, N>(ring + i * slot_bytes, false, H);
            ring_clear<YT, V, N>(ring + i * slot_bytes + xb, !has_prev, H);
        }
    int pt = blockIdx.x;  // the next row to copy
    auto prefetch = [&](int slot) {
        if constexpr (kRing) {
            if (pt < a.T) {
                ring_copy<XT, V, N>(ring + slot * slot_bytes, (const XT*)a.x + (size_t)pt * a.ldx + c0, H);
                if (has_prev) ring_copy<YT, V, N>(ring + slot * slot_bytes + xb, (const YT*)a.y + (size_t)pt * a.ldy + c0, H);
            }
            cp_async_commit();
            pt += gridDim.x;
        }
    };
    float2 b[N * V / 2], q[N * V / 2];
    // one row's copies, then the parameters (they would wait behind a full ring), then the other slots'
    for (int k = 0; k == 0 || k < stages - 1; ++k) {
        prefetch(k);
        if (k) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            float2 f[V / 2];
            if (has_prev) load_branch<V>(a, c, f);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) b[i * V / 2 + j] = f[j];
            if (has_next) load_columns<V>(a.pre, c, H, f);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) q[i * V / 2 + j] = f[j];
        }
    }
    int slot = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        Piece<XT, V> rx[N];
        Piece<YT, V> ry[N];
        if constexpr (kRing) {
            cp_async_wait(stages);
            // into the slot of the row before this one, which this thread has read
            if (stages > 1) prefetch(slot == 0 ? stages - 1 : slot - 1);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            take<XT, V, kRing>(rx[i], true, i, ring + slot * slot_bytes, (const XT*)a.x + (size_t)t * a.ldx + c0, H);
            take<YT, V, kRing>(ry[i], has_prev, i, ring + slot * slot_bytes + xb, (const YT*)a.y + (size_t)t * a.ldy + c0, H);
        }
        if (kRing && stages == 1) prefetch(0);
        slot = slot + 1 >= stages ? 0 : slot + 1;
        if (has_prev) {
            float w = a.token ? a.token[t] : 1.0f;
            if (post) w *= row_scale<YT, V, N, single>(ry, H, inv, a.eps_post, red[0], red64[0]);
            XT* xo = (XT*)a.xo + (size_t)t * a.ldxo + c0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 x[V / 2], y[V / 2];
                rx[i].get(x);
                ry[i].get(y);
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                    x[j] = __ffma2_rn(b[i * V / 2 + j], __fmul2_rn(both(w), y[j]), __fmul2_rn(both(a.xs), x[j]));
                rx[i].set(x);  // from here on as stored: what a later read of x_out sees
                const int left = H - (int)(i * blockDim.x + threadIdx.x) * V;
                if (left > 0) rx[i].store(xo + i * blockDim.x * V, left);
                if (left < V) {
                    if (left <= 0) rx[i].zero();
                    else if constexpr (V == 2) rx[i].b.zero();
                }
            }
        }
        if (has_next) {
            const float2 r = both(row_scale<XT, V, N, single>(rx, H, inv, a.eps_pre, red[1], red64[1]));
            NT* no = (NT*)a.n + (size_t)t * a.ldn + c0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 v[V / 2];
                rx[i].get(v);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) v[j] = __fmul2_rn(__fmul2_rn(v[j], r), q[i * V / 2 + j]);
                const int left = H - (int)(i * blockDim.x + threadIdx.x) * V;
                Piece<NT, V> out;
                out.set(v);
                if (left > 0) out.store(no + i * blockDim.x * V, left);
            }
        }
        if constexpr (single) break;
        // with one sum a row, the next row's would use the same buffer
        if (!(has_prev && post && has_next)) __syncthreads();
    }
}

// Rows too wide for registers: the same sums over columns that a thread reads
// again from memory (x_out again after it stored it, by the same thread). In fp64:
// a thread adds up to 128 columns one after another, which in fp32 could lose 60
// steps of 2^-24 of 1 / rms where the narrow rows' sums lose 18 at most (1.5 us of
// the 96 for 1024 x 16384 bf16, whose bytes take 21: columns are read one at a time).
template <typename XT, typename YT, typename NT>
__global__ void __launch_bounds__(1024) block_norm_wide_kernel(NormArgs a) {
    __shared__ double red64[2][32];
    const int t = blockIdx.x, H = a.H;
    const XT* x = (const XT*)a.x + (size_t)t * a.ldx;
    const YT* y = (const YT*)a.y + (size_t)t * a.ldy;
    XT* xo = a.has_prev ? (XT*)a.xo + (size_t)t * a.ldxo : nullptr;
    double ss[1] = {0.0};
    if (a.has_prev) {
        float rho = 1.0f;
        if (a.post_norm) {
            for (int c = threadIdx.x; c < H; c += blockDim.x) {
                Raw<YT, 1> r;
                r.load(y + c);
                float v[1];
                r.get(v);
                ss[0] += (double)v[0] * v[0];
            }
            block_sum<double, 1>(ss, red64[0]);
            rho = rms_scale(ss[0], H, a.eps_post);
        }
        const float scale = a.ys * (a.token ? a.token[t] : 1.0f);
        ss[0] = 0.0;
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            Raw<XT, 1> rx;
            Raw<YT, 1> ry;
            rx.load(x + c);
            ry.load(y + c);
            float vx[1], vy[1];
            rx.get(vx);
            ry.get(vy);
            vx[0] = fmaf(scale * gain(a.gate, c), vy[0] * rho * gain(a.post, c), a.xs * vx[0]);
            rx.set(vx);
            rx.store(xo + c);
            rx.get(vx);
            ss[0] += (double)vx[0] * vx[0];
        }
        x = xo;
    } else {
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            Raw<XT, 1> rx;
            rx.load(x + c);
            float v[1];
            rx.get(v);
            ss[0] += (double)v[0] * v[0];
        }
    }
    if (!a.has_next) return;
    block_sum<double, 1>(ss, red64[1]);
    const float r = rms_scale(ss[0], H, a.eps_pre);
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
        Raw<XT, 1> rx;
        rx.load(x + c);
        float v[1];
        rx.get(v);
        v[0] = v[0] * r * gain(a.pre, c);
        Raw<NT, 1> out;
        out.set(v);
        out.store((NT*)a.n + (size_t)t * a.ldn + c);
    }
}

// ---------------------------------------------------------------------------
// Backward. With sh = s r and yh = y rho (the normalised rows), b = ys g p:
//   ds = dxo + r (q dn - sh m1), m1 = mean(sh q dn)      dx = xs ds      dq = sum_t sh dn
//   dy = rho (u b ds - yh m2),   m2 = mean(yh u b ds)    du = sum_c b yh ds
//   A  = sum_t u yh ds, of which dp = ys g A and dg = ys p A
// m2 and du need ds only in sums, and ds is linear in three of them, so one
// round of six sums a row is enough:
//   s^2, s q dn, y^2, b y dxo, b y q dn, b y s:   sum b yh ds = rho (S3 + r (S4 - r m1 S5)).
// Without `next` no output depends on s: it is 0 then, so that infinities and NaN in
// x_out do not show.
// A block keeps dq and A of its threads' columns over its rows in registers;
// sum_parts_kernel adds the blocks'.
// At 2048 x 6144 bf16 (151 MB): 36 us, of which the rows take 24 (6.3 TB/s), the
// start 3, the blocks' sums 6. With half the columns a thread and twice the warps
// the rows took 50: what every warp repeats for a row (sums, factors, addresses)
// is more than half of its instructions then.
// ---------------------------------------------------------------------------
// post: without the post norm dy has no part of y, not even 0 y, so that infinities
// and NaN in y do not show. (As a condition on every value it took 0.3 to 0.5 us of
// the 36, and 3 % where rows are read by columns.)
template <typename XT, typename YT, typename NT, int V, int N, bool post>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const NormArgs a) {
    __shared__ float red[2][16 * 8];
    __shared__ double red64[32 * 6];
    extern __shared__ __align__(16) unsigned char ring_mem[];
    constexpr bool kRing = V >= 4;
    const int H = a.H, stages = a.stages, c0 = threadIdx.x * V;
    const bool has_prev = a.has_prev, has_next = a.has_next, has_o = a.dxo != nullptr;
    uint32_t yo = 0, oo = 0, no = 0, slot_bytes = 0;  // offsets of y, dxo and dn in a slot
    if constexpr (kRing) {
        yo = ring_bytes<XT, V, N>();
        oo = yo + ring_bytes<YT, V, N>();
        no = oo + ring_bytes<XT, V, N>();
        slot_bytes = no + ring_bytes<NT, V, N>();
    }
    const uint32_t ring = smem_addr(ring_mem);
    if constexpr (kRing)
        for (int i = 0; i < stages; ++i) {
            ring_clear<XT, V, N>(ring + i * slot_bytes, !has_next, H);
            ring_clear<YT, V, N>(ring + i * slot_bytes + yo, !has_prev, H);
            ring_clear<XT, V, N>(ring + i * slot_bytes + oo, !has_o, H);
            ring_clear<NT, V, N>(ring + i * slot_bytes + no, !has_next, H);
        }
    int pt = blockIdx.x;  // the next row to copy
    auto prefetch = [&](int slot) {
        if constexpr (kRing) {
            if (pt < a.T) {
                const uint32_t at = ring + slot * slot_bytes;
                if (has_next) ring_copy<XT, V, N>(at, (const XT*)a.x + (size_t)pt * a.ldx + c0, H);
                if (has_prev) ring_copy<YT, V, N>(at + yo, (const YT*)a.y + (size_t)pt * a.ldy + c0, H);
                if (has_o) ring_copy<XT, V, N>(at + oo, (const XT*)a.dxo + (size_t)pt * a.lddxo + c0, H);
                if (has_next) ring_copy<NT, V, N>(at + no, (const NT*)a.dn + (size_t)pt * a.lddn + c0, H);
            }
            cp_async_commit();
            pt += gridDim.x;
        }
    };
    grid_next();  // sum_parts_kernel may start: it waits for this one's end itself
    constexpr int P = V / 2;
    float2 b[N * P], q[N * P], dq[N * P], A[N * P];
    prefetch(0);  // one row, then the parameters: behind a full ring (21 MB) they came 3 us later
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        float2 f[P], g[P];
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = g[j] = both(0.0f);
        if (has_prev) load_branch<V>(a, c, f);
        if (has_next) load_columns<V>(a.pre, c, H, g);
#pragma unroll
        for (int j = 0; j < P; ++j) b[i * P + j] = f[j], q[i * P + j] = g[j], dq[i * P + j] = A[i * P + j] = both(0.0f);
    }
    for (int i = 1; i < stages - 1; ++i) prefetch(i);
    // V = 2: the next row's columns are loaded while a row is worked on, where the registers allow it
    constexpr bool kAhead = V == 2 && N <= 4;
    constexpr int kKept = kRing ? 1 : N;
    Piece<XT, V> rs[kKept], ro[kKept];
    Piece<YT, V> ry[kKept];
    Piece<NT, V> rn[kKept];
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            take<XT, V, false>(rs[i], has_next, i, 0, (const XT*)a.x + (size_t)t * a.ldx + c0, H);
            take<YT, V, false>(ry[i], has_prev, i, 0, (const YT*)a.y + (size_t)t * a.ldy + c0, H);
            take<XT, V, false>(ro[i], has_o, i, 0, (const XT*)a.dxo + (size_t)t * a.lddxo + c0, H);
            take<NT, V, false>(rn[i], has_next, i, 0, (const NT*)a.dn + (size_t)t * a.lddn + c0, H);
        }
    };
    if constexpr (kAhead) fetch(blockIdx.x);
    int slot = 0, flip = 0;
    const float inv = 1.0f / (float)H;
    const bool tiny_s = has_next && a.eps_pre < 1e-12f, tiny_y = post && a.eps_post < 1e-12f;  // see sum_ok
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        if constexpr (kRing) {
            cp_async_wait(stages);
            // into the slot of the row before this one, which this thread has read
            if (stages > 1) prefetch(slot == 0 ? stages - 1 : slot - 1);
        }
        const uint32_t at = ring + slot * slot_bytes;
        slot = slot + 1 >= stages ? 0 : slot + 1;
        // Wide pieces are read from the ring in every pass over the row; single columns stay in registers
        // (as values where the next row's are being loaded).
        float2 ks[kAhead ? N : 1], ky[kAhead ? N : 1], ko[kAhead ? N : 1], kn[kAhead ? N : 1];
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                rs[i].get(reinterpret_cast<float2(&)[P]>(ks[i]));
                ry[i].get(reinterpret_cast<float2(&)[P]>(ky[i]));
                ro[i].get(reinterpret_cast<float2(&)[P]>(ko[i]));
                rn[i].get(reinterpret_cast<float2(&)[P]>(kn[i]));
            }
            if (t + (int)gridDim.x < a.T) fetch(t + gridDim.x);
        }
        auto row = [&](int i, int pass, float2 (&s)[P], float2 (&y)[P], float2 (&o)[P], float2 (&n)[P]) {
            if constexpr (kAhead) {
                s[0] = ks[i], y[0] = ky[i], o[0] = ko[i], n[0] = kn[i];
            } else {
                const int k = kRing ? 0 : i;
                if (kRing || pass == 0) {
                    take<XT, V, kRing>(rs[k], has_next, i, at, (const XT*)a.x + (size_t)t * a.ldx + c0, H);
                    take<YT, V, kRing>(ry[k], has_prev, i, at + yo, (const YT*)a.y + (size_t)t * a.ldy + c0, H);
                    take<XT, V, kRing>(ro[k], has_o, i, at + oo, (const XT*)a.dxo + (size_t)t * a.lddxo + c0, H);
                    take<NT, V, kRing>(rn[k], has_next, i, at + no, (const NT*)a.dn + (size_t)t * a.lddn + c0, H);
                }
                rs[k].get(s);
                ry[k].get(y);
                ro[k].get(o);
                rn[k].get(n);
            }
        };
        const float u = a.token ? a.token[t] : 1.0f;
        float2 acc[6];
#pragma unroll
        for (int j = 0; j < 6; ++j) acc[j] = both(0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 s[P], n[P], y[P], o[P];
            row(i, 0, s, y, o, n);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 qn = __fmul2_rn(q[i * P + j], n[j]), by = __fmul2_rn(b[i * P + j], y[j]);
                acc[0] = __ffma2_rn(s[j], s[j], acc[0]);
                acc[1] = __ffma2_rn(s[j], qn, acc[1]);
                acc[2] = __ffma2_rn(y[j], y[j], acc[2]);
                acc[3] = __ffma2_rn(by, o[j], acc[3]);
                acc[4] = __ffma2_rn(by, qn, acc[4]);
                acc[5] = __ffma2_rn(by, s[j], acc[5]);
            }
        }
        float v[6];
#pragma unroll
        for (int j = 0; j < 6; ++j) v[j] = acc[j].x + acc[j].y;
        block_sums(v, red[flip]);
        flip ^= 1;
        float r = 0.0f, m1 = 0.0f, rho = 1.0f, du;
        // every sum finite and in range (not so with NaN), no squares lost that eps does not hide
        const float big = fabsf(v[0]) + fabsf(v[1]) + fabsf(v[2]) + fabsf(v[3]) + fabsf(v[4]) + fabsf(v[5]);
        if (big <= 3e37f && !(tiny_s && v[0] < 1e-24f) && !(tiny_y && v[2] < 1e-24f)) {
            if (has_next) {
                r = rsqrtf(fmaf(v[0], inv, a.eps_pre));
                m1 = v[1] * r * inv;
            }
            if (post) rho = rsqrtf(fmaf(v[2], inv, a.eps_post));
            du = rho * fmaf(r, fmaf(-r * m1, v[5], v[4]), v[3]);
        } else {  // a row beyond fp32's range (or not finite): the same sums in fp64
            double w[6] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float2 s2[P], n2[P], y2[P], o2[P];
                row(i, 1, s2, y2, o2, n2);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int k = j / 2;
                    const bool hi = j & 1;
                    const double s = hi ? s2[k].y : s2[k].x, y = hi ? y2[k].y : y2[k].x, o = hi ? o2[k].y : o2[k].x;
                    const double qn = (double)(hi ? q[i * P + k].y : q[i * P + k].x) * (hi ? n2[k].y : n2[k].x);
                    const double by = (double)(hi ? b[i * P + k].y : b[i * P + k].x) * y;
                    w[0] += s * s;
                    w[1] += s * qn;
                    w[2] += y * y;
                    w[3] += by * o;
                    w[4] += by * qn;
                    w[5] += by * s;
                }
            }
            block_sum<double, 6>(w, red64);
            __syncthreads();  // the next such row reuses red64
            double rd = 0.0, md = 0.0, pd = 1.0;
            if (has_next) {
                rd = 1.0 / sqrt(w[0] / H + (double)a.eps_pre);
                md = w[1] * rd / H;
            }
            if (post) pd = 1.0 / sqrt(w[2] / H + (double)a.eps_post);
            r = (float)rd;
            m1 = (float)md;
            rho = (float)pd;
            du = (float)(pd * (w[3] + rd * (w[4] - rd * md * w[5])));
        }
        if (a.dtoken && threadIdx.x == 0) a.dtoken[t] = du;
        const float2 m2 = both(post ? -u * du * inv : 0.0f), r2 = both(r), m1n = both(-m1), rho2 = both(rho), u2 = both(u);
        XT* dx = (XT*)a.dx + (size_t)t * a.lddx + c0;
        YT* dy = (YT*)a.dy + (size_t)t * a.lddy + c0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 s[P], n[P], y[P], o[P];
            row(i, 1, s, y, o, n);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = i * P + j;
                const float2 sh = __fmul2_rn(s[j], r2), yh = __fmul2_rn(y[j], rho2);
                dq[k] = __ffma2_rn(sh, n[j], dq[k]);
                o[j] = __ffma2_rn(r2, __ffma2_rn(sh, m1n, __fmul2_rn(q[k], n[j])), o[j]);  // ds
                const float2 uo = __fmul2_rn(u2, o[j]);
                A[k] = __ffma2_rn(yh, uo, A[k]);
                y[j] = __fmul2_rn(b[k], uo);
                if constexpr (post) y[j] = __fmul2_rn(rho2, __ffma2_rn(yh, m2, y[j]));
                o[j] = __fmul2_rn(both(a.xs), o[j]);
            }
            const int left = H - (int)(i * blockDim.x + threadIdx.x) * V;
            if (left <= 0) continue;
            if (a.dx) {
                Piece<XT, V> out;
                out.set(o);
                out.store(dx + i * blockDim.x * V, left);
            }
            if (a.dy) {
                Piece<YT, V> out;
                out.set(y);
                out.store(dy + i * blockDim.x * V, left);
            }
        }
        if (stages == 1) prefetch(0);
    }
    if (a.part) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            float* out = a.part + (size_t)blockIdx.x * 2 * H + c;
            if constexpr (kRing) {
                if (c >= H) continue;
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    const float2 x0 = dq[i * P + j], x1 = dq[i * P + j + 1], y0 = A[i * P + j], y1 = A[i * P + j + 1];
                    *reinterpret_cast<float4*>(out + 2 * j) = make_float4(x0.x, x0.y, x1.x, x1.y);
                    *reinterpret_cast<float4*>(out + H + 2 * j) = make_float4(y0.x, y0.y, y1.x, y1.y);
                }
            } else {
                if (c < H) {
                    out[0] = dq[i].x;
                    out[H] = A[i].x;
                }
                if (c + 1 < H) {
                    out[1] = dq[i].y;
                    out[H + 1] = A[i].y;
                }
            }
        }
    }
}

// Rows too wide for registers: the columns are read again in each round, one at
// a time, and the sums over a block's rows grow in its part of the workspace.
// 1024 x 16384 bf16 593 us, where its bytes take 31: latency of single loads at 16
// warps an SM.
template <typename XT, typename YT, typename NT>
__global__ void __launch_bounds__(1024) block_norm_backward_wide_kernel(NormArgs a) {
    __shared__ double red64[2][32 * 3];
    const int H = a.H;
    float* part = a.part ? a.part + (size_t)blockIdx.x * 2 * H : nullptr;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float u = a.token ? a.token[t] : 1.0f;
        const bool first = t == (int)blockIdx.x;
        auto row = [&](int c, float& s, float& y, float& n, float& o) {
            s = y = n = o = 0.0f;
            float v[1];
            Raw<XT, 1> rx;
            rx.load((const XT*)a.x + (size_t)t * a.ldx + c);
            rx.get(v);
            s = v[0];
            if (a.dxo) {
                rx.load((const XT*)a.dxo + (size_t)t * a.lddxo + c);
                rx.get(v);
                o = v[0];
            }
            if (a.has_prev) {
                Raw<YT, 1> ry;
                ry.load((const YT*)a.y + (size_t)t * a.ldy + c);
                ry.get(v);
                y = v[0];
            }
            if (a.has_next) {
                Raw<NT, 1> rn;
                rn.load((const NT*)a.dn + (size_t)t * a.lddn + c);
                rn.get(v);
                n = v[0];
            }
        };
        double w[3] = {0.0, 0.0, 0.0};
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            float s, y, n, o;
            row(c, s, y, n, o);
            w[0] += (double)s * s;
            w[1] += (double)s * gain(a.pre, c) * n;
            w[2] += (double)y * y;
        }
        block_sum<double, 3>(w, red64[0]);
        const float r = rms_scale(w[0], H, a.eps_pre);  // without next it and s, sh and m1 show in no output
        const float m1 = (float)(w[1] * (double)r / H);
        const float rho = a.post_norm ? rms_scale(w[2], H, a.eps_post) : 1.0f;
        double v[1] = {0.0};
        float m2 = 0.0f;
        for (int round = 0; round < 2; ++round) {
            for (int c = threadIdx.x; c < H; c += blockDim.x) {
                float s, y, n, o;
                row(c, s, y, n, o);
                const float b = a.has_prev ? gain(a.gate, c) * (a.ys * gain(a.post, c)) : 0.0f;
                const float sh = s * r;
                if (a.has_next) o = fmaf(r, fmaf(-sh, m1, gain(a.pre, c) * n), o);
                const float yh = y * rho;
                if (round == 0) {
                    v[0] += (double)b * yh * o;
                    if (part) {
                        part[c] = first ? sh * n : fmaf(sh, n, part[c]);
                        part[H + c] = first ? u * yh * o : fmaf(u * yh, o, part[H + c]);
                    }
                } else {  // every input of this column has been read: dx and dy may be inputs
                    float f[1] = {a.xs * o};
                    if (a.dx) {
                        Raw<XT, 1> out;
                        out.set(f);
                        out.store((XT*)a.dx + (size_t)t * a.lddx + c);
                    }
                    if (a.dy) {
                        f[0] = u * b * o;
                        if (a.post_norm) f[0] = rho * fmaf(-yh, m2, f[0]);
                        Raw<YT, 1> out;
                        out.set(f);
                        out.store((YT*)a.dy + (size_t)t * a.lddy + c);
                    }
                }
            }
            if (round == 0) {
                block_sum<double, 1>(v, red64[1]);
                if (a.dtoken && threadIdx.x == 0) a.dtoken[t] = (float)v[0];
                m2 = a.post_norm ? (float)(u * v[0] / H) : 0.0f;
            }
        }
    }
}

// The gains' and the gate's gradients from the blocks' sums, added in block
// order: 32 columns and 16 runs of blocks a block, ten loads of a run in flight.
__global__ void __launch_bounds__(512) sum_parts_kernel(const NormArgs a, int n, float* dpre, float* dpost, float* dgate) {
    __shared__ float sh[16][32];
    grid_wait();
    const int H = a.H, which = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    if (which == 0 ? !dpre : !dpost && !dgate) return;
    const int per = (n + 15) / 16, b0 = g * per, b1 = min(n, b0 + per);
    float acc = 0.0f;
    for (int b = b0; b < b1 && c < H; b += 10) {
        float v[10];
#pragma unroll
        for (int j = 0; j < 10; ++j) v[j] = b + j < b1 ? __ldcg(a.part + ((size_t)(b + j) * 2 + which) * H + c) : 0.0f;
#pragma unroll
        for (int j = 0; j < 10; ++j) acc += v[j];
    }
    sh[g][threadIdx.x & 31] = acc;
    __syncthreads();
    if (g != 0 || c >= H) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) acc += sh[i][threadIdx.x];
    if (which == 0) {
        dpre[c] = acc;
        return;
    }
    acc *= a.ys;
    if (dpost) dpost[c] = acc * (a.gate ? a.gate[c] : 1.0f);
    if (dgate) dgate[c] = acc * (a.post ? a.post[c] : 1.0f);
}

constexpr int kSms = 148;
// Up to here a block takes one row without the ring. In us, without it and with it: 148 rows of 6144 bf16 3.8 and
// 4.4, 149 rows (two blocks on some SM) 5.9 and 5.1; of fp32 4.8 and 6.0, then 7.0 and 7.0, and with 2048 rows 55 and
// 41. Rows of 512 to 2048 columns differ by 0.5 at most up to 300 rows; from 444 on fp32 rows would take up to 1.5
// less without the ring (2048 x 512: 4.5 and 6.0), 2048 bf16 rows of 2048 columns 1.6 more.
constexpr int kSingleRows = kSms;
// V, N and threads for rows of H columns, up to 512 threads; N == 0: too wide
// for registers. V: columns that all rows take at a time (8 or 4), or 2.
struct Shape {
    int V, N, threads;
};
Shape shape_of(int H, int V) {
    const int n = (H + V - 1) / V;
    for (int N : {1, 2, 4, 8}) {
        if (N * V > 16) break;
        const int th = ((n + N - 1) / N + 31) / 32 * 32;
        if (th <= 512) return {V, N, th};
    }
    return {V, 0, 512};
}

// Blocks that share an SM: as many as their registers let (80 a thread
// forward, 128 backward), at most 16 (8: each block leaves its sums).
int blocks_per_sm(int threads, bool fwd) {
    const int n = (fwd ? kForwardThreads : 512) / threads, most = fwd ? 16 : 8;
    return n < 1 ? 1 : n > most ? most : n;
}
// Blocks of a persistent launch over T rows. The workspace's size depends on
// it: it must not depend on the alignment of a call's rows.
int grid_of(int T, int H, bool fwd) {
    const int g = kSms * blocks_per_sm(shape_of(H, H % 8 == 0 ? 8 : H % 4 == 0 ? 4 : 2).threads, fwd);
    return T < g ? T : g;
}
constexpr size_t kRingBytes = 200 * 1024;  // of an SM's shared memory
// Ring slots of `row` bytes (at most 128 KB) that fit beside the other blocks of an SM.
int stages_of(size_t row, int threads, int rows, bool fwd) {
    const size_t n = kRingBytes / blocks_per_sm(threads, fwd) / row;
    return n < 1 || rows < 2 ? 1 : n > 4 ? 4 : (int)n;
}

using B = __nv_bfloat16;
using Kernel = void (*)(NormArgs);

cudaError_t launch_rows(Kernel k, NormArgs& a, const Shape& s, size_t col_bytes, int grid, bool fwd, cudaStream_t st) {
    const size_t row = s.V >= 4 && s.N ? col_bytes * s.V * s.N * s.threads : 0;
    a.stages = row ? stages_of(row, s.threads, (a.T + grid - 1) / grid, fwd) : 0;
    const size_t smem = a.stages * row;
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_shared(k, kRingBytes);
        if (e != cudaSuccess) return e;
    }
    return launch(k, grid, s.threads, smem, st, false, a);
}

template <typename XT, typename YT, typename NT>
cudaError_t forward_typed(NormArgs& a, int V, cudaStream_t st) {
    constexpr bool narrow = sizeof(XT) + sizeof(YT) + sizeof(NT) == 6;  // all bf16
    const int n = (a.H + V - 1) / V;
    if (a.T <= kSingleRows && V >= 4 && n <= kForwardThreads * (8 / V)) {
        const int N = 8 / V, th = ((n + N - 1) / N + 31) / 32 * 32;
        if constexpr (narrow)
            if (V == 8) return launch(block_norm_kernel<XT, YT, NT, 8, 1, true>, a.T, th, 0, st, false, a);
        return launch(block_norm_kernel<XT, YT, NT, 4, 2, true>, a.T, th, 0, st, false, a);
    }
    const Shape s = shape_of(a.H, V);
    Kernel k = block_norm_wide_kernel<XT, YT, NT>;
    if (s.N && V == 8) {
        if constexpr (narrow) k = s.N == 1 ? block_norm_kernel<XT, YT, NT, 8, 1, false> : block_norm_kernel<XT, YT, NT, 8, 2, false>;
    } else if (s.N && V == 4) {
        k = s.N == 1   ? block_norm_kernel<XT, YT, NT, 4, 1, false>
            : s.N == 2 ? block_norm_kernel<XT, YT, NT, 4, 2, false>
                       : block_norm_kernel<XT, YT, NT, 4, 4, false>;
    } else if (s.N) {
        k = s.N == 1   ? block_norm_kernel<XT, YT, NT, 2, 1, false>
            : s.N == 2 ? block_norm_kernel<XT, YT, NT, 2, 2, false>
            : s.N == 4 ? block_norm_kernel<XT, YT, NT, 2, 4, false>
                       : block_norm_kernel<XT, YT, NT, 2, 8, false>;
    }
    return launch_rows(k, a, s, sizeof(XT) + sizeof(YT), s.N ? grid_of(a.T, a.H, true) : a.T, true, st);
}

template <typename XT, typename YT, typename NT, bool post>
cudaError_t backward_typed(NormArgs& a, int V, cudaStream_t st) {
    constexpr bool narrow = sizeof(XT) + sizeof(YT) + sizeof(NT) == 6;
    const Shape s = shape_of(a.H, V);
    Kernel k = block_norm_backward_wide_kernel<XT, YT, NT>;
    if (s.N && V == 8) {
        if constexpr (narrow) k = s.N == 1 ? block_norm_backward_kernel<XT, YT, NT, 8, 1, post> : block_norm_backward_kernel<XT, YT, NT, 8, 2, post>;
    } else if (s.N && V == 4) {
        k = s.N == 1   ? block_norm_backward_kernel<XT, YT, NT, 4, 1, post>
            : s.N == 2 ? block_norm_backward_kernel<XT, YT, NT, 4, 2, post>
                       : block_norm_backward_kernel<XT, YT, NT, 4, 4, post>;
    } else if (s.N) {
        k = s.N == 1   ? block_norm_backward_kernel<XT, YT, NT, 2, 1, post>
            : s.N == 2 ? block_norm_backward_kernel<XT, YT, NT, 2, 2, post>
            : s.N == 4 ? block_norm_backward_kernel<XT, YT, NT, 2, 4, post>
                       : block_norm_backward_kernel<XT, YT, NT, 2, 8, post>;
    }
    return launch_rows(k, a, s, 2 * sizeof(XT) + sizeof(YT) + sizeof(NT), grid_of(a.T, a.H, false), false, st);
}

template <bool fwd>
cudaError_t by_type(NormArgs& a, coli_dtype xt, coli_dtype yt, coli_dtype nt, int V, cudaStream_t st) {
    auto go = [&](auto x, auto y, auto n) {
        if constexpr (fwd) return forward_typed<decltype(x), decltype(y), decltype(n)>(a, V, st);
        else return a.post_norm ? backward_typed<decltype(x), decltype(y), decltype(n), true>(a, V, st)
                                : backward_typed<decltype(x), decltype(y), decltype(n), false>(a, V, st);
    };
    auto with_n = [&](auto x, auto y) { return nt == COLI_F32 ? go(x, y, float()) : go(x, y, B()); };
    auto with_y = [&](auto x) { return yt == COLI_F32 ? with_n(x, float()) : with_n(x, B()); };
    return xt == COLI_F32 ? with_y(float()) : with_y(B());
}

// Columns that all of a call's rows and arrays take at a time: 8 (all bf16), 4,
// or 2 read one by one. m: the matrices, NULL where absent.
int columns_of(const NormArgs& a, std::initializer_list<const Mat*> m) {
    if (((uintptr_t)a.pre | (uintptr_t)a.post | (uintptr_t)a.gate) & 15u) return 2;
    for (int V : {8, 4}) {
        bool ok = true;
        for (const Mat* x : m) ok = ok && (!x || (x->takes(V) && (V == 4 || x->t == COLI_BF16)));
        if (ok) return V;
    }
    return 2;
}

#define REQUIRE(cond, msg)                                \
    do {                                                  \
        if (!(cond)) return block_fail(COLI_EINVAL, msg); \
    } while (0)

void set_params(NormArgs& a, const coli_block_params* prev, const coli_block_params* next) {
    a.has_prev = prev != nullptr;
    a.has_next = next != nullptr;
    a.xs = 1.0f;
    if (prev) {
        a.post = prev->post_gain;
        a.gate = prev->gate;
        a.xs = prev->x_scale;
        a.ys = prev->y_scale;
        a.eps_post = prev->eps;
        a.post_norm = prev->post_norm;
    }
    if (next) {
        a.pre = next->pre_gain;
        a.eps_pre = next->eps;
    }
}

coli_status check_sizes(const coli_block_params* prev, const coli_block_params* next, int T, int H, int device) {
    REQUIRE(prev || next, "prev and next are both NULL");
    for (const coli_block_params* p : {prev, next})
        if (p)
            if (const char* m = check_block_params(p)) return block_fail(COLI_EINVAL, m);
    REQUIRE(T >= 0 && T <= kBlockMaxTokens, "n_tokens must be in [0, 2^20]");
    REQUIRE(H >= 1 && H <= kBlockMaxHidden, "hidden must be in [1, 65536]");
    REQUIRE(device >= 0, "no such CUDA device");
    return COLI_OK;
}

struct Span {
    const void* p;
    size_t n;
};
const char* outputs_overlap(const Span* out, int no, const Span* in, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return "an output overlaps an input";
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return "two outputs overlap";
    }
    return nullptr;
}

}  // namespace

const char* check_block_params(const coli_block_params* p) {
    if (!(p->eps >= 0.0f)) return "eps must be >= 0";
    if (p->post_norm != 0 && p->post_norm != 1) return "post_norm must be 0 or 1";
    if (p->post_gain && !p->post_norm) return "post_gain given without post_norm";
    if (((uintptr_t)p->pre_gain | (uintptr_t)p->post_gain | (uintptr_t)p->gate) & 3u) return "gains and gate must be 4-byte aligned";
    return nullptr;
}

coli_status block_norm_launch(const coli_block_params* prev, const coli_block_params* next, const Mat* x, const Mat* y,
                              const Mat* x_out, const Mat* n, const float* token_gate, int T, int H, cudaStream_t st) {
    NormArgs a{};
    a.T = T;
    a.H = H;
    set_params(a, prev, next);
    a.x = x->p;
    a.ldx = x->stride;
    a.token = token_gate;
    if (prev) {
        a.y = y->p;
        a.ldy = y->stride;
        a.xo = x_out->p ? const_cast<void*>(x_out->p) : nullptr;
        a.ldxo = x_out->stride;
    }
    if (next) {
        a.n = const_cast<void*>(n->p);
        a.ldn = n->stride;
    }
    const int V = columns_of(a, {x, prev ? y : nullptr, prev ? x_out : nullptr, next ? n : nullptr});
    const cudaError_t e = by_type<true>(a, x->t, prev ? y->t : x->t, next ? n->t : x->t, V, st);
    return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "block norm");
}

}  // namespace coli

using namespace coli;

#define CHECK_MAT(m, name)                                                                                        \
    do {                                                                                                          \
        if (const char* _m = check_mat(m, name " is NULL", name "_stride is smaller than hidden",                  \
                                       name " is not aligned to its element"))                                    \
            return block_fail(COLI_EINVAL, _m);                                                                   \
    } while (0)

COLI_API coli_status coli_block_norm(const coli_block_params* prev, const coli_block_params* next, const void* x,
                                     coli_dtype x_dtype, int64_t x_stride, const void* y, coli_dtype y_dtype,
                                     int64_t y_stride, const float* token_gate, void* x_out, int64_t x_out_stride,
                                     void* n, coli_dtype n_dtype, int64_t n_stride, int T, int H, int device,
                                     coli_stream stream) {
    coli_status s = check_sizes(prev, next, T, H, device);
    if (s != COLI_OK) return s;
    REQUIRE(dtype_ok(x_dtype) && (!prev || dtype_ok(y_dtype)) && (!next || dtype_ok(n_dtype)),
            "dtypes must be COLI_F32 or COLI_BF16");
    REQUIRE(prev || (!y && !x_out && !token_gate), "y, x_out and token_gate need prev");
    REQUIRE(next || !n, "n needs next");
    REQUIRE(((uintptr_t)token_gate & 3u) == 0, "token_gate must be 4-byte aligned");
    if (T == 0) return COLI_OK;
    const Mat mx{x, x_dtype, T, H, x_stride}, my{y, y_dtype, T, H, y_stride}, mo{x_out, x_dtype, T, H, x_out_stride},
        mn{n, n_dtype, T, H, n_stride};
    CHECK_MAT(mx, "x");
    Span ins[8];
    int ni = 0;
    const size_t hb = (size_t)H * 4;
    if (prev) {
        CHECK_MAT(my, "y");
        CHECK_MAT(mo, "x_out");
        REQUIRE(same(mo, mx) || !overlap(mo, mx), "x_out and x overlap");
        REQUIRE(!overlap(mo, my), "x_out and y overlap");
        ins[ni++] = {prev->post_gain, hb};
        ins[ni++] = {prev->gate, hb};
        ins[ni++] = {token_gate, (size_t)T * 4};
    }
    if (next) {
        CHECK_MAT(mn, "n");
        REQUIRE(!overlap(mn, mx), "n and x overlap");
        REQUIRE(!prev || same(mn, my) || !overlap(mn, my), "n and y overlap");
        REQUIRE(!prev || !overlap(mn, mo), "n and x_out overlap");
        ins[ni++] = {next->pre_gain, hb};
    }
    const Span outs[] = {{x_out, prev ? mo.bytes() : 0}, {n, next ? mn.bytes() : 0}};
    for (int i = 0; i < 2; ++i)
        if (const char* m = outputs_overlap(outs + i, 1, ins, ni)) return block_fail(COLI_EINVAL, m);
    DeviceGuard guard(device);
    REQUIRE(guard.ok, "no such CUDA device");
    return block_norm_launch(prev, next, &mx, &my, &mo, &mn, token_gate, T, H, (cudaStream_t)stream);
}

COLI_API int64_t coli_block_norm_workspace(int T, int H) {
    if (T < 0 || T > kBlockMaxTokens || H < 1 || H > kBlockMaxHidden) return -1;
    return (int64_t)grid_of(T, H, false) * 2 * H * 4;
}

COLI_API coli_status coli_block_norm_backward(const coli_block_params* prev, const coli_block_params* next,
                                              const void* x_out, coli_dtype x_dtype, int64_t x_out_stride, const void* y,
                                              coli_dtype y_dtype, int64_t y_stride, const float* token_gate,
                                              const void* dx_out, int64_t dx_out_stride, const void* dn,
                                              coli_dtype n_dtype, int64_t dn_stride, void* dx, int64_t dx_stride,
                                              void* dy, int64_t dy_stride, float* dpre_gain, float* dpost_gain,
                                              float* dgate, float* dtoken_gate, void* work, int64_t work_bytes, int T,
                                              int H, int device, coli_stream stream) {
    coli_status st = check_sizes(prev, next, T, H, device);
    if (st != COLI_OK) return st;
    REQUIRE(dtype_ok(x_dtype) && (!prev || dtype_ok(y_dtype)) && (!next || dtype_ok(n_dtype)),
            "dtypes must be COLI_F32 or COLI_BF16");
    REQUIRE(prev || (!y && !dy && !token_gate && !dpost_gain && !dgate && !dtoken_gate),
            "y, dy, the gates and their gradients need prev");
    REQUIRE(next || (!dn && !dpre_gain), "dn and dpre_gain need next");
    REQUIRE(!dpost_gain || prev->post_norm, "dpost_gain needs post_norm");
    REQUIRE((((uintptr_t)token_gate | (uintptr_t)dpre_gain | (uintptr_t)dpost_gain | (uintptr_t)dgate |
              (uintptr_t)dtoken_gate) & 3u) == 0,
            "gains, gates and their gradients must be 4-byte aligned");
    const bool want = dpre_gain || dpost_gain || dgate;
    const int64_t need = want ? coli_block_norm_workspace(T, H) : 0;
    REQUIRE(need == 0 || (work && work_bytes >= need), "work is smaller than coli_block_norm_workspace");
    REQUIRE(need == 0 || ((uintptr_t)work & 15u) == 0, "work must be 16-byte aligned");
    const Mat ms{x_out, x_dtype, T, H, x_out_stride}, my{y, y_dtype, T, H, y_stride},
        mo{dx_out, x_dtype, T, H, dx_out_stride}, mn{dn, n_dtype, T, H, dn_stride}, mdx{dx, x_dtype, T, H, dx_stride},
        mdy{dy, y_dtype, T, H, dy_stride};
    CHECK_MAT(ms, "x_out");
    if (prev) CHECK_MAT(my, "y");
    if (next) CHECK_MAT(mn, "dn");
    if (dx_out) CHECK_MAT(mo, "dx_out");
    if (dx) CHECK_MAT(mdx, "dx");
    if (dy) CHECK_MAT(mdy, "dy");
    const Mat* in[4] = {&ms, prev ? &my : nullptr, dx_out ? &mo : nullptr, next ? &mn : nullptr};
    for (int i = 0; i < 4; ++i) {
        if (!in[i]) continue;
        if (dx) REQUIRE(((i == 0 || i == 2) && same(mdx, *in[i])) || !overlap(mdx, *in[i]), "dx overlaps an input");
        if (dy) REQUIRE(((i == 1 || i == 3) && same(mdy, *in[i])) || !overlap(mdy, *in[i]), "dy overlaps an input");
    }
    if (dx && dy) REQUIRE(!overlap(mdx, mdy), "dx and dy overlap");
    const size_t hb = (size_t)H * 4, tb = (size_t)T * 4;
    const Span ins[] = {{prev ? prev->post_gain : nullptr, hb}, {prev ? prev->gate : nullptr, hb}, {token_gate, tb},
                        {next ? next->pre_gain : nullptr, hb}};
    const Span outs[] = {{dx, dx ? mdx.bytes() : 0}, {dy, dy ? mdy.bytes() : 0}, {dpre_gain, hb}, {dpost_gain, hb},
                         {dgate, hb}, {dtoken_gate, tb}, {need ? work : nullptr, (size_t)need}};
    if (const char* m = outputs_overlap(outs + 2, 5, ins, 4)) return block_fail(COLI_EINVAL, m);
    for (int i = 0; i < 2; ++i) {
        if (const char* m = outputs_overlap(outs + i, 1, ins, 4)) return block_fail(COLI_EINVAL, m);
        for (int j = 2; j < 7; ++j) REQUIRE(!overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n), "two outputs overlap");
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 2; j < 7; ++j)
            REQUIRE(!in[i] || !overlap(in[i]->p, in[i]->bytes(), outs[j].p, outs[j].n), "an output overlaps an input");
    DeviceGuard guard(device);
    REQUIRE(guard.ok, "no such CUDA device");
    cudaStream_t s = (cudaStream_t)stream;
    NormArgs a{};
    a.T = T;
    a.H = H;
    set_params(a, prev, next);
    a.x = x_out;
    a.ldx = x_out_stride;
    a.y = y;
    a.ldy = y_stride;
    a.token = token_gate;
    a.dxo = dx_out;
    a.lddxo = dx_out_stride;
    a.dn = dn;
    a.lddn = dn_stride;
    a.dx = dx;
    a.lddx = dx_stride;
    a.dy = dy;
    a.lddy = dy_stride;
    a.dtoken = dtoken_gate;
    a.part = want ? (float*)work : nullptr;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        const int V = columns_of(a, {&ms, in[1], in[2], in[3], dx ? &mdx : nullptr, dy ? &mdy : nullptr});
        e = by_type<false>(a, x_dtype, prev ? y_dtype : x_dtype, next ? n_dtype : x_dtype, V, s);
        if (e != cudaSuccess) return block_cuda_fail(e, "block norm backward");
    }
    if (!want) return COLI_OK;
    e = launch(sum_parts_kernel, dim3((H + 31) / 32, 2), 512, 0, s, T > 0, a, grid_of(T, H, false), dpre_gain, dpost_gain, dgate);
    return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "block norm backward: gains");
}

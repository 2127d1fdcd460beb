// dispatch.cu -- tokens sorted by expert and back, with their gradients
// (coli_moe_dispatch, coli_moe_combine and their backward calls).
#include "block.cuh"

#define COLI_API extern "C" __attribute__((visibility("default")))

namespace coli {
namespace {

// ---------------------------------------------------------------------------
// The sort. Slots i = t * K + k are cut into chunks, one block each. A block
// ranks its chunk: every warp owns a run of consecutive slots, counts its
// experts, and the slot's row is
//   offsets[e] + (slots of e in earlier chunks) + (in earlier warps) + (before it in its warp),
// so the order is (t, k) order and nothing depends on timing.
// ---------------------------------------------------------------------------
constexpr int kSms = 148;
constexpr int kRankThreads = 1024;
constexpr int kRankWarps = kRankThreads / 32;
constexpr int kChunkSlots = 2048;  // slots of a chunk, until there are kMaxChunks of them
constexpr int kMaxChunks = 64;

struct Chunks {
    int size, n;
};
Chunks chunks_of(int64_t slots) {
    const int64_t per = (slots + kMaxChunks - 1) / kMaxChunks;
    Chunks c;
    c.size = (int)(per > kChunkSlots ? (per + 1023) / 1024 * 1024 : kChunkSlots);
    c.n = (int)((slots + c.size - 1) / c.size);
    if (c.n < 1) c.n = 1;
    return c;
}

// Slots of each expert in each chunk.
__global__ void __launch_bounds__(kRankThreads) dispatch_count_kernel(const int32_t* ids, int n, int E, int chunk,
                                                                      int32_t* hist) {
    __shared__ int32_t h[1024];
    for (int e = threadIdx.x; e < E; e += kRankThreads) h[e] = 0;
    __syncthreads();
    const int end = min(n, (int)(blockIdx.x + 1) * chunk);
    for (int i = blockIdx.x * chunk + threadIdx.x; i < end; i += kRankThreads) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(h + e, 1);  // an integer count: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRankThreads) hist[(size_t)blockIdx.x * E + e] = h[e];
    grid_next();
}

// Exclusive prefix of v over the block's kRankThreads threads, and the total.
__device__ __forceinline__ int block_scan(int v, int32_t* sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + s - v;
}

// Dynamic shared memory: wcnt [kRankWarps][E], then sums [32].
__global__ void __launch_bounds__(kRankThreads) dispatch_rank_kernel(const int32_t* ids, int n, int E, int chunk,
                                                                     const int32_t* hist, int32_t* counts,
                                                                     int32_t* offsets, int32_t* pos, int32_t* slot) {
    extern __shared__ int32_t sh[];
    int32_t* wcnt = sh;
    int32_t* sums = sh + kRankWarps * E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
    const int per = chunk / kRankWarps;  // a multiple of 32
    const int w0 = c0 + warp * per, w1 = min(c1, w0 + per);
    for (int i = threadIdx.x; i < kRankWarps * E; i += kRankThreads) wcnt[i] = 0;
    __syncthreads();
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < w1 ? ids[i] : -1;
        if ((unsigned)e < (unsigned)E) atomicAdd(wcnt + warp * E + e, 1);  // an integer count: the order does not matter
    }
    __syncthreads();
    int mine = 0;  // this chunk's slots of expert e = threadIdx.x, its warps' counts made exclusive
    if (threadIdx.x < E) {
#pragma unroll 8
        for (int w = 0; w < kRankWarps; ++w) {
            const int v = wcnt[w * E + threadIdx.x];
            wcnt[w * E + threadIdx.x] = mine;
            mine += v;
        }
    }
    int total = 0, before = 0;  // over all chunks; over the chunks before this one
    grid_wait();
    if (threadIdx.x < E)
#pragma unroll 8
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const int v = hist[(size_t)b * E + threadIdx.x];
            if (b < (int)blockIdx.x) before += v;
            total += v;
        }
    int all;
    const int off = block_scan(total, sums, &all);
    if (threadIdx.x < E) {
#pragma unroll 8
        for (int w = 0; w < kRankWarps; ++w) wcnt[w * E + threadIdx.x] += off + before;
        if (blockIdx.x == 0) {
            counts[threadIdx.x] = total;
            offsets[threadIdx.x] = off;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = all;
    __syncthreads();
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < w1 ? ids[i] : -1;
        const unsigned m = __match_any_sync(0xffffffffu, e);
        const bool held = (unsigned)e < (unsigned)E;
        int q = -1;
        if (held) {
            q = wcnt[warp * E + e] + __popc(m & ((1u << lane) - 1u));
            slot[q] = i;
        }
        if (i < w1) pos[i] = q;
        __syncwarp();
        if (held && lane == __ffs(m) - 1) wcnt[warp * E + e] += __popc(m);
        __syncwarp();
    }
    for (int i = max(c0, all) + threadIdx.x; i < c1; i += kRankThreads) slot[i] = -1;  // behind the last expert
    grid_next();
}

constexpr int kMaxExperts = 1024;
size_t rank_smem(int E) { return sizeof(int32_t) * ((size_t)kRankWarps * E + 32); }

// ---------------------------------------------------------------------------
// The same sort in one launch for up to kClusterSlots slots: a cluster of eight
// blocks, a chunk each, which read each other's counts from shared memory. A
// warp's first 64 slots stay in registers between the two passes. With the rows
// (256 columns of bf16), dispatch takes 12.2 us for 28000 slots where the two
// launches above take 12.4, but 12.9 against 12.1 for 32768 and 17.9 against 14.5
// for 48000: eight blocks are then too few. Bound by its steps' latency: for
// 16384 slots 1.2 us until the slots are read, 2 of barrier (1.5 of them the
// warps' matching), 1.5 of the others' counts and the scan, 1.1 of placing.
// Counting by matching lanes too, as placing does, took 2.4 us more.
// ---------------------------------------------------------------------------
constexpr int kCluster = 8;
constexpr int kClusterSlots = 24576;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A word of block `rank`'s shared memory, at the place that `p` has in this block's.
__device__ __forceinline__ int32_t cluster_read(const int32_t* p, int rank) {
    uint32_t a;
    int32_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__global__ void __launch_bounds__(kRankThreads, 1) dispatch_sort_kernel(const int32_t* ids, int n, int E, int chunk,
                                                                        int32_t* counts, int32_t* offsets, int32_t* pos,
                                                                        int32_t* slot) {
    extern __shared__ int32_t sh[];  // wcnt [kRankWarps][E], tot [E], sums [32]
    int32_t *wcnt = sh, *tot = sh + kRankWarps * E, *sums = tot + E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = blockIdx.x;
    grid_next();  // the rows kernel may start: it waits for this one's end itself
    const int c0 = min(n, rank * chunk), c1 = min(n, c0 + chunk), per = chunk / kRankWarps;
    const int w0 = c0 + warp * per, w1 = min(c1, w0 + per);
    auto fetch = [&](int i) {
        const int e = i < w1 ? ids[i] : -1;
        return (unsigned)e < (unsigned)E ? e : -1;
    };
    int kept[2];
    kept[0] = fetch(w0 + lane);
    kept[1] = fetch(w0 + 32 + lane);
    for (int i = threadIdx.x; i < kRankWarps * E; i += kRankThreads) wcnt[i] = 0;
    __syncthreads();
    auto count = [&](int e) {
        if (e >= 0) atomicAdd(wcnt + warp * E + e, 1);  // an integer count: the order does not matter
    };
    count(kept[0]);
    if (per > 32) count(kept[1]);
    for (int i0 = w0 + 64; i0 < w0 + per; i0 += 32) count(fetch(i0 + lane));
    __syncthreads();
    int mine = 0, c[kRankWarps];
    if (threadIdx.x < E) {
#pragma unroll
        for (int w = 0; w < kRankWarps; ++w) c[w] = wcnt[w * E + threadIdx.x];
#pragma unroll
        for (int w = 0; w < kRankWarps; ++w) {
            const int v = c[w];
            c[w] = mine;
            mine += v;
        }
        tot[threadIdx.x] = mine;
    }
    cluster_arrive();
    // the lanes with the same expert, while the other blocks come
    const unsigned same[2] = {__match_any_sync(0xffffffffu, kept[0]), __match_any_sync(0xffffffffu, kept[1])};
    cluster_wait();
    int total = 0, before = 0;  // over all chunks; over the chunks before this one
    if (threadIdx.x < E) {
#pragma unroll
        for (int b = 0; b < kCluster; ++b) {
            const int v = cluster_read(tot + threadIdx.x, b);
            if (b < rank) before += v;
            total += v;
        }
    }
    cluster_arrive();  // (no block leaves before the others have read its counts)
    int all;
    const int off = block_scan(total, sums, &all);
    if (threadIdx.x < E) {
#pragma unroll
        for (int w = 0; w < kRankWarps; ++w) wcnt[w * E + threadIdx.x] = c[w] + off + before;
        if (rank == 0) {
            counts[threadIdx.x] = total;
            offsets[threadIdx.x] = off;
        }
    }
    if (rank == 0 && threadIdx.x == 0) offsets[E] = all;
    __syncthreads();
    auto place = [&](int i, int e, unsigned m) {
        int q = -1;
        if (e >= 0) {
            q = wcnt[warp * E + e] + __popc(m & ((1u << lane) - 1u));
            slot[q] = i;
        }
        if (i < w1) pos[i] = q;
        __syncwarp();
        if (e >= 0 && lane == __ffs(m) - 1) wcnt[warp * E + e] += __popc(m);
        __syncwarp();
    };
    place(w0 + lane, kept[0], same[0]);
    if (per > 32) place(w0 + 32 + lane, kept[1], same[1]);
    for (int i0 = w0 + 64; i0 < w0 + per; i0 += 32) {
        const int e = fetch(i0 + lane);
        place(i0 + lane, e, __match_any_sync(0xffffffffu, e));
    }
    for (int i = max(c0, all) + threadIdx.x; i < c1; i += kRankThreads) slot[i] = -1;  // behind the last expert
    cluster_wait();
}

// Pieces of V columns that a thread takes, a block's width apart: narrow pieces
// would spend more loads on the positions than on the rows.
template <int V>
constexpr int kPieces = V >= 4 ? 1 : V == 2 ? 2 : 4;

// rows[pos[t][k]] = x[t]: a thread reads its columns of a token once and writes
// them K times. Bound by the K rows a token writes: 2048 x 8 x 6144 bf16 (226 MB)
// in 36 us, 6.3 TB/s. Rows that start on odd values are written 2 bytes at a
// time, at half that rate.
template <typename XT, typename RT, int V>
__global__ void __launch_bounds__(128) dispatch_rows_kernel(const XT* x, int64_t ldx, const int32_t* pos, int K, int H,
                                                            RT* rows, int64_t ldr) {
    constexpr int N = kPieces<V>;
    const int t = blockIdx.x, step = blockDim.x * V;
    const int c0 = blockIdx.y * N * step + threadIdx.x * V;
    Raw<RT, V> out[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Raw<XT, V> in;
        in.zero();
        if (c0 + i * step < H) in.load(x + (size_t)t * ldx + c0 + i * step);  // x is older than the sort: read while that still runs
        float v[V];
        in.get(v);
        out[i].set(v);
    }
    grid_wait();
    for (int k = 0; k < K; ++k) {
        const int q = pos[(size_t)t * K + k];
        if (q < 0) continue;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c0 + i * step < H) out[i].store(rows + (size_t)q * ldr + c0 + i * step);
    }
}

// y[t] = base[t] + sum_k w[t][k] rows[pos[t][k]], the rows of eight slots in
// flight at a time. Bound by the K rows a token reads: 8192 x 8 x 6144 bf16 (906
// MB) in 140 us, 6.5 TB/s. Rows of odd bf16 width wait for their 2-byte loads: a
// quarter of that rate; loading all of a thread's pieces first was slower still
// (fewer warps fit).
template <typename RT, typename YT, int V>
__global__ void __launch_bounds__(128, sizeof(RT) == 4 ? 8 : 6) gather_sum_kernel(const int32_t* pos, const float* w, bool skip_zero, int K, const RT* rows,
                                                         int64_t ldr, int n_rows, int H, const YT* base, int64_t ldb,
                                                         YT* y, int64_t ldy) {
    grid_wait();
    constexpr int N = kPieces<V>;
    const int t = blockIdx.x, step = blockDim.x * V;
    const int c0 = blockIdx.y * N * step + threadIdx.x * V;
    if (c0 >= H) return;
    float acc[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Raw<YT, V> b;
        b.zero();
        if (base && c0 + i * step < H) b.load(base + (size_t)t * ldb + c0 + i * step);
        b.get(acc[i]);
    }
    for (int k0 = 0; k0 < K; k0 += 8) {
        float wk[8];
        int q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = k0 + j;
            q[j] = k < K ? pos[(size_t)t * K + k] : -1;
            if (q[j] >= n_rows) q[j] = -1;
            wk[j] = q[j] >= 0 && w ? w[(size_t)t * K + k] : 1.0f;
            if (skip_zero && wk[j] == 0.0f) q[j] = -1;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = c0 + i * step;
            if (N > 1 && c >= H) break;
            Raw<RT, V> r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (q[j] >= 0) r[j].load(rows + (size_t)q[j] * ldr + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (q[j] < 0) continue;
                float v[V];
                r[j].get(v);
#pragma unroll
                for (int l = 0; l < V; ++l) acc[i][l] = fmaf(wk[j], v[l], acc[i][l]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Raw<YT, V> out;
        out.set(acc[i]);
        if (c0 + i * step < H) out.store(y + (size_t)t * ldy + c0 + i * step);
    }
}

// drows[pos] = w dy[t], dweights = dot(dy[t], rows[pos]): one block per token,
// eight slots at a time, dy read once. Bound by the K rows a token reads and
// writes: 2048 x 8 x 6144 bf16 (428 MB) in 71 us, 6 TB/s.
template <typename RT, typename YT, int V>
__global__ void __launch_bounds__(256) combine_backward_kernel(const int32_t* pos, const float* w, int K, const YT* dy,
                                                               int64_t ldy, int H, const RT* rows, int64_t ldr,
                                                               int64_t n_rows, RT* drows, int64_t ldd, float* dw) {
    __shared__ float red[2][32 * 8];
    const int t = blockIdx.x;
    int flip = 0;
    for (int k0 = 0; k0 < K; k0 += 8) {
        int64_t q[8];
        float wk[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = k0 + j;
            q[j] = k < K ? pos[(size_t)t * K + k] : -1;
            if (q[j] >= n_rows) q[j] = -1;
            wk[j] = q[j] >= 0 && drows ? w[(size_t)t * K + k] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x * V; c < H; c += blockDim.x * V) {
            Raw<YT, V> g;
            g.load(dy + (size_t)t * ldy + c);
            Raw<RT, V> r[8];
            if (dw)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (q[j] >= 0) r[j].load(rows + (size_t)q[j] * ldr + c);
            float gv[V];
            g.get(gv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (q[j] < 0) continue;
                if (dw) {
                    float v[V];
                    r[j].get(v);
#pragma unroll
                    for (int i = 0; i < V; ++i) dot[j] = fmaf(gv[i], v[i], dot[j]);
                }
                if (drows) {
                    float v[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = wk[j] * gv[i];
                    Raw<RT, V> out;
                    out.set(v);
                    out.store(drows + (size_t)q[j] * ldd + c);
                }
            }
        }
        if (dw) {
            block_sum<float, 8>(dot, red[flip]);
            flip ^= 1;
            if (threadIdx.x == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k0 + j < K) dw[(size_t)t * K + k0 + j] = dot[j];
        }
    }
}

// Threads of a block, and blocks of `pieces` pieces a thread, for rows of H
// columns: blocks of up to 128 threads that share the columns evenly (combine of
// 8192 x 8 x 6144 bf16 140 us, 6.5 TB/s; with up to 256 threads 146 us).
struct Tiles {
    int threads, n;
};
Tiles tiles_of(int H, int V, int pieces = 1) {
    const int all = (H + V * pieces - 1) / (V * pieces), n = (all + 127) / 128;
    return {((all + n - 1) / n + 31) / 32 * 32, n};
}

// The largest of 8, 4, 2 and 1 columns a thread that all these matrices take,
// `rows` (the experts' side, most of the bytes) first; 8 only where they are
// bf16 (of fp32, a warp's two accesses would lie 32 bytes apart and read every
// 32-byte sector twice).
int columns_of(const Mat& rows, const Mat& b, const Mat* c = nullptr) {
    for (int V : {8, 4, 2}) {
        if (V == 8 && rows.t != COLI_BF16) continue;
        if (rows.takes(V) && b.takes(V) && (!c || c->takes(V))) return V;
    }
    return 1;
}

template <typename XT, typename RT>
cudaError_t dispatch_rows(const Mat& x, const int32_t* pos, int T, int K, const Mat& rows, cudaStream_t st) {
    const int V = columns_of(rows, x);
    const Tiles g = tiles_of(x.cols, V, V >= 4 ? 1 : V == 2 ? 2 : 4);  // kPieces
    auto k = V == 4   ? dispatch_rows_kernel<XT, RT, 4>
             : V == 2 ? dispatch_rows_kernel<XT, RT, 2>
                      : dispatch_rows_kernel<XT, RT, 1>;
    if constexpr (sizeof(RT) == 2)
        if (V == 8) k = dispatch_rows_kernel<XT, RT, 8>;
    return launch(k, dim3(T, g.n), g.threads, 0, st, true, (const XT*)x.p, x.stride, pos, K, x.cols, (RT*)rows.p,
                  rows.stride);
}

template <typename RT, typename YT>
cudaError_t gather_sum(const int32_t* pos, const float* w, bool skip_zero, int T, int K, const Mat& rows, const Mat* base,
                       const Mat& y, cudaStream_t st, bool dependent) {
    const int V = columns_of(rows, y, base);
    const Tiles g = tiles_of(y.cols, V, V >= 4 ? 1 : V == 2 ? 2 : 4);  // kPieces
    auto k = V == 4   ? gather_sum_kernel<RT, YT, 4>
             : V == 2 ? gather_sum_kernel<RT, YT, 2>
                      : gather_sum_kernel<RT, YT, 1>;
    if constexpr (sizeof(RT) == 2)
        if (V == 8) k = gather_sum_kernel<RT, YT, 8>;
    return launch(k, dim3(T, g.n), g.threads, 0, st, dependent, pos, w, skip_zero, K, (const RT*)rows.p, rows.stride,
                  (int)(rows.rows < INT32_MAX ? rows.rows : INT32_MAX), y.cols, (const YT*)(base ? base->p : nullptr), base ? base->stride : 0, (YT*)y.p, y.stride);
}

template <typename RT, typename YT>
cudaError_t combine_backward(const int32_t* pos, const float* w, int T, int K, const Mat& dy, const Mat& rows,
                             const Mat* drows, float* dw, cudaStream_t st) {
    const int V = dw ? columns_of(rows, dy, drows) : columns_of(*drows, dy);
    auto k = V == 4   ? combine_backward_kernel<RT, YT, 4>
             : V == 2 ? combine_backward_kernel<RT, YT, 2>
                      : combine_backward_kernel<RT, YT, 1>;
    if constexpr (sizeof(RT) == 2)
        if (V == 8) k = combine_backward_kernel<RT, YT, 8>;
    // many tokens: small blocks, whose sums hold up fewer loads (2048 x 8 x 6144 bf16 71 us against 75 with
    // 256 threads, x 4 x 2048 19 against 27); few: one token's columns at once (64 x 8 x 6144 5.8 against 8.3)
    const int all = ((dy.cols + V - 1) / V + 31) / 32 * 32, most = T >= 4 * kSms ? 128 : 256;
    return launch(k, T, all < most ? all : most, 0, st, false, pos, w, K, (const YT*)dy.p, dy.stride, dy.cols,
                  (const RT*)rows.p, rows.stride, rows.rows, (RT*)(drows ? drows->p : nullptr), drows ? drows->stride : 0, dw);
}

// ---------------------------------------------------------------------------
// Few slots (decoding): one launch does all. A block takes a token and a tile
// of columns, and finds the rows of its K slots by comparing them with every
// slot: row = number of slots of lower experts, and of the same expert before
// it. The last block writes the counts, the offsets and the slots' tail. One
// launch costs the caller 2 us less than two, and one token's 8 rows of 6144 take
// 2.5 us of the GPU's time instead of 4.9.
// ---------------------------------------------------------------------------
constexpr int kFewSlots = 1024;
constexpr int kFewThreads = 256;

struct Few {
    const int32_t* ids;
    int T, K, E, H, move;
    int64_t ldx, ldr;
    int32_t *counts, *offsets, *pos, *slot;
};

template <typename XT, typename RT, int V>
__global__ void __launch_bounds__(kFewThreads) dispatch_few_kernel(const Few a, const XT* x, RT* rows) {
    constexpr int kEach = kFewSlots / kFewThreads;
    __shared__ int32_t found[32][kFewThreads / 32];
    __shared__ int32_t hist[1024], sums[32];
    const int n = a.T * a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x, c = (blockIdx.y * kFewThreads + threadIdx.x) * V;
    int32_t e[kEach];  // slots threadIdx.x, + 256, ..; E: an empty slot
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = threadIdx.x + j * kFewThreads;
        const int id = i < n ? a.ids[i] : a.E;
        e[j] = (unsigned)id < (unsigned)a.E ? id : a.E;
    }
    if (t == a.T) {
        if (blockIdx.y) return;
        for (int i = threadIdx.x; i < a.E; i += kFewThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (e[j] < a.E) atomicAdd(hist + e[j], 1);  // an integer count: the order does not matter
        __syncthreads();
        int v[4], own = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = threadIdx.x * 4 + j;
            v[j] = i < a.E ? hist[i] : 0;
            own += v[j];
        }
        int s = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        int off = s - own, all = 0;
        for (int w = 0; w < kFewThreads / 32; ++w) {
            if (w < warp) off += sums[w];
            all += sums[w];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = threadIdx.x * 4 + j;
            if (i < a.E) {
                a.counts[i] = v[j];
                a.offsets[i] = off;
            }
            off += v[j];
        }
        if (threadIdx.x == 0) a.offsets[a.E] = all;
        for (int i = all + threadIdx.x; i < n; i += kFewThreads) a.slot[i] = -1;
        return;
    }
    Raw<XT, V> in;
    in.zero();
    if (a.move && c < a.H) in.load(x + (size_t)t * a.ldx + c);
    for (int k = 0; k < a.K; ++k) {
        const int i = t * a.K + k, id = a.ids[i];
        int before = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int at = threadIdx.x + j * kFewThreads;
            before += e[j] < id || (e[j] == id && at < i);
        }
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) found[k][warp] = before;
    }
    __syncthreads();
    float f[V];
    in.get(f);
    Raw<RT, V> out;
    out.set(f);
    for (int k = 0; k < a.K; ++k) {
        const int i = t * a.K + k, id = a.ids[i];
        const bool held = (unsigned)id < (unsigned)a.E;
        int q = 0;
#pragma unroll
        for (int w = 0; w < kFewThreads / 32; ++w) q += found[k][w];
        if (held && a.move && c < a.H) out.store(rows + (size_t)q * a.ldr + c);
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            a.pos[i] = held ? q : -1;
            if (held) a.slot[q] = i;
        }
    }
}

template <typename XT, typename RT>
cudaError_t dispatch_few(const Few& a, const Mat& x, const Mat& rows, cudaStream_t st) {
    const int V = a.move ? columns_of(rows, x) : 4;
    auto k = V == 4   ? dispatch_few_kernel<XT, RT, 4>
             : V == 2 ? dispatch_few_kernel<XT, RT, 2>
                      : dispatch_few_kernel<XT, RT, 1>;
    if constexpr (sizeof(RT) == 2)
        if (V == 8) k = dispatch_few_kernel<XT, RT, 8>;
    const int tiles = a.move ? (a.H + V * kFewThreads - 1) / (V * kFewThreads) : 1;
    return launch(k, dim3(a.T + 1, tiles), kFewThreads, 0, st, false, a, (const XT*)x.p, (RT*)rows.p);
}

const char* check_slots(int T, int K) {
    if (T < 0 || T > kBlockMaxTokens) return "n_tokens must be in [0, 2^20]";
    if (K < 1 || K > 32) return "top_k must be in [1, 32]";
    if ((int64_t)T * K > kBlockMaxSlots) return "n_tokens * top_k must be at most 2^24";
    return nullptr;
}

#define TRY_ARG(expr)                                                   \
    do {                                                                \
        if (const char* _m = (expr)) return block_fail(COLI_EINVAL, _m); \
    } while (0)
#define REQUIRE(cond, msg)                                  \
    do {                                                    \
        if (!(cond)) return block_fail(COLI_EINVAL, msg);   \
    } while (0)

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

coli_status check_combine(const int32_t* pos, int T, int K, const Mat& rows, bool need_rows, int H) {
    TRY_ARG(check_slots(T, K));
    REQUIRE(H >= 1 && H <= kBlockMaxHidden, "hidden must be in [1, 65536]");
    REQUIRE(dtype_ok(rows.t), "rows_dtype must be COLI_F32 or COLI_BF16");
    REQUIRE(rows.rows >= 0, "n_rows must be >= 0");
    if (T == 0) return COLI_OK;
    REQUIRE(pos, "pos is NULL");
    REQUIRE(aligned4(pos), "pos must be 4-byte aligned");
    if (need_rows)
        TRY_ARG(check_mat(rows, "rows is NULL", "rows_stride is smaller than hidden", "rows is not aligned to its element"));
    return COLI_OK;
}

// y = base + sum of rows: dispatch_backward and combine.
coli_status gather_entry(const int32_t* pos, const float* w, int T, int K, const Mat& rows, const void* base,
                         int64_t base_stride, const Mat& y, int device, cudaStream_t st) {
    coli_status s = check_combine(pos, T, K, rows, true, y.cols);
    if (s != COLI_OK) return s;
    REQUIRE(dtype_ok(y.t), "the output's dtype must be COLI_F32 or COLI_BF16");
    REQUIRE(device >= 0, "no such CUDA device");
    if (T == 0) return COLI_OK;
    TRY_ARG(check_mat(y, "the output is NULL", "the output's stride is smaller than hidden",
                      "the output is not aligned to its element"));
    const Mat b{base, y.t, T, y.cols, base_stride};
    if (base) {
        TRY_ARG(check_mat(b, "", "base_stride is smaller than hidden", "base is not aligned to its element"));
        REQUIRE(same(b, y) || !overlap(b, y), "base and the output overlap");
    }
    REQUIRE(!overlap(rows, y), "rows and the output overlap");
    REQUIRE(!overlap(y.p, y.bytes(), pos, (size_t)T * K * 4), "pos and the output overlap");
    REQUIRE(!overlap(y.p, y.bytes(), w, (size_t)T * K * 4), "weights and the output overlap");
    DeviceGuard guard(device);
    REQUIRE(guard.ok, "no such CUDA device");
    cudaError_t e = launch_gather_sum(pos, w, false, T, K, rows, base ? &b : nullptr, y, st, false);
    return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "combine");
}

}  // namespace

cudaError_t launch_gather_sum(const int32_t* pos, const float* w, bool skip_zero, int T, int K, const Mat& rows,
                              const Mat* base, const Mat& y, cudaStream_t st, bool dependent) {
    const bool rf = rows.t == COLI_F32, yf = y.t == COLI_F32;
    using B = __nv_bfloat16;
    if (rf) return yf ? gather_sum<float, float>(pos, w, skip_zero, T, K, rows, base, y, st, dependent)
                      : gather_sum<float, B>(pos, w, skip_zero, T, K, rows, base, y, st, dependent);
    return yf ? gather_sum<B, float>(pos, w, skip_zero, T, K, rows, base, y, st, dependent)
              : gather_sum<B, B>(pos, w, skip_zero, T, K, rows, base, y, st, dependent);
}

}  // namespace coli

using namespace coli;

COLI_API int64_t coli_moe_dispatch_workspace(int T, int K, int E) {
    if (check_slots(T, K) || E < 1 || E > kMaxExperts) return -1;
    const int64_t n = (int64_t)T * K, chunks = (n + kChunkSlots - 1) / kChunkSlots;
    // the most chunks that so many slots or fewer are cut into (just above kMaxChunks * kChunkSlots slots there are
    // fewer, larger ones)
    return n > kClusterSlots ? (chunks < kMaxChunks ? chunks : kMaxChunks) * E * 4 : 0;
}

COLI_API coli_status coli_moe_dispatch(const int32_t* ids, int T, int K, int E, const void* x, coli_dtype x_dtype,
                                       int64_t x_stride, int hidden, int32_t* counts, int32_t* offsets, int32_t* pos,
                                       int32_t* slot, void* rows, coli_dtype rows_dtype, int64_t rows_stride,
                                       int64_t n_rows, void* work, int64_t work_bytes, int device, coli_stream stream) {
    TRY_ARG(check_slots(T, K));
    REQUIRE(E >= 1 && E <= kMaxExperts, "n_experts must be in [1, 1024]");
    REQUIRE(counts && offsets, "counts or offsets is NULL");
    REQUIRE(T == 0 || (ids && pos && slot), "ids, pos or slot is NULL");
    REQUIRE(aligned4(ids) && aligned4(counts) && aligned4(offsets) && aligned4(pos) && aligned4(slot),
            "int32 arrays must be 4-byte aligned");
    REQUIRE((x == nullptr) == (rows == nullptr) || T == 0, "x and rows: both or neither");
    REQUIRE(device >= 0, "no such CUDA device");
    const size_t n = (size_t)T * K;
    const Mat mx{x, x_dtype, T, hidden, x_stride}, mr{rows, rows_dtype, n_rows, hidden, rows_stride};
    const bool move = x && rows && T > 0;
    if (move) {
        REQUIRE(hidden >= 1 && hidden <= kBlockMaxHidden, "hidden must be in [1, 65536]");
        REQUIRE(dtype_ok(x_dtype) && dtype_ok(rows_dtype), "dtypes must be COLI_F32 or COLI_BF16");
        REQUIRE(n_rows >= (int64_t)n, "n_rows must be at least n_tokens * top_k");
        TRY_ARG(check_mat(mx, "x is NULL", "x_stride is smaller than hidden", "x is not aligned to its element"));
        TRY_ARG(check_mat(mr, "rows is NULL", "rows_stride is smaller than hidden", "rows is not aligned to its element"));
        REQUIRE(!overlap(mx, mr), "x and rows overlap");
    }
    const int64_t need = n > kClusterSlots ? (int64_t)chunks_of((int64_t)n).n * E * 4 : 0;
    REQUIRE(need == 0 || (work && work_bytes >= need), "work is smaller than coli_moe_dispatch_workspace");
    REQUIRE(((uintptr_t)work & 15u) == 0, "work must be 16-byte aligned");
    const void* outs[] = {counts, offsets, pos, slot, move ? rows : nullptr, need ? work : nullptr};
    const size_t len[] = {(size_t)E * 4, (size_t)(E + 1) * 4, n * 4, n * 4, move ? mr.bytes() : 0, (size_t)need};
    for (int i = 0; i < 6; ++i) {
        REQUIRE(!overlap(outs[i], len[i], ids, n * 4), "an output overlaps ids");
        REQUIRE(i == 4 || !move || !overlap(outs[i], len[i], x, mx.bytes()), "an output overlaps x");
        for (int j = 0; j < i; ++j) REQUIRE(!overlap(outs[i], len[i], outs[j], len[j]), "two outputs overlap");
    }
    DeviceGuard guard(device);
    REQUIRE(guard.ok, "no such CUDA device");
    cudaStream_t st = (cudaStream_t)stream;
    const Chunks c = chunks_of((int64_t)n);
    cudaError_t e = cudaSuccess;
    using B = __nv_bfloat16;
    if (n <= kFewSlots) {
        const Few f{ids, T, K, E, hidden, move, x_stride, rows_stride, counts, offsets, pos, slot};
        if (!move || x_dtype == COLI_F32)
            e = !move || rows_dtype == COLI_F32 ? dispatch_few<float, float>(f, mx, mr, st) : dispatch_few<float, B>(f, mx, mr, st);
        else
            e = rows_dtype == COLI_F32 ? dispatch_few<B, float>(f, mx, mr, st) : dispatch_few<B, B>(f, mx, mr, st);
        return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "dispatch");
    }
    if (n <= kClusterSlots) {
        const int chunk = (int)((n + kCluster * kRankThreads - 1) / (kCluster * kRankThreads)) * kRankThreads;
        const size_t smem = rank_smem(E) + (size_t)E * 4;
        e = allow_shared(dispatch_sort_kernel, rank_smem(kMaxExperts) + kMaxExperts * 4);
        if (e != cudaSuccess) return block_cuda_fail(e, "dispatch: shared memory");
        e = launch_clusters(kCluster, dispatch_sort_kernel, kCluster, kRankThreads, smem, st, false, ids, (int)n, E, chunk,
                            counts, offsets, pos, slot);
        if (e != cudaSuccess) return block_cuda_fail(e, "dispatch: sort");
    } else {
        e = launch(dispatch_count_kernel, c.n, kRankThreads, 0, st, false, ids, (int)n, E, c.size, (int32_t*)work);
        if (e != cudaSuccess) return block_cuda_fail(e, "dispatch: count");
        const size_t smem = rank_smem(E);
        e = allow_shared(dispatch_rank_kernel, rank_smem(kMaxExperts));
        if (e != cudaSuccess) return block_cuda_fail(e, "dispatch: shared memory");
        e = launch(dispatch_rank_kernel, c.n, kRankThreads, smem, st, true, ids, (int)n, E, c.size, (const int32_t*)work,
                   counts, offsets, pos, slot);
        if (e != cudaSuccess) return block_cuda_fail(e, "dispatch: rank");
    }
    if (!move) return COLI_OK;
    if (x_dtype == COLI_F32)
        e = rows_dtype == COLI_F32 ? dispatch_rows<float, float>(mx, pos, T, K, mr, st)
                                   : dispatch_rows<float, B>(mx, pos, T, K, mr, st);
    else
        e = rows_dtype == COLI_F32 ? dispatch_rows<B, float>(mx, pos, T, K, mr, st)
                                   : dispatch_rows<B, B>(mx, pos, T, K, mr, st);
    return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "dispatch: rows");
}

COLI_API coli_status coli_moe_dispatch_backward(const int32_t* pos, int T, int K, const void* drows,
                                                coli_dtype rows_dtype, int64_t rows_stride, int64_t n_rows, int hidden,
                                                const void* base, int64_t base_stride, void* dx, coli_dtype dx_dtype,
                                                int64_t dx_stride, int device, coli_stream stream) {
    return gather_entry(pos, nullptr, T, K, Mat{drows, rows_dtype, n_rows, hidden, rows_stride}, base, base_stride,
                        Mat{dx, dx_dtype, T, hidden, dx_stride}, device, (cudaStream_t)stream);
}

COLI_API coli_status coli_moe_combine(const int32_t* pos, const float* weights, int T, int K, const void* rows,
                                      coli_dtype rows_dtype, int64_t rows_stride, int64_t n_rows, int hidden,
                                      const void* base, int64_t base_stride, void* y, coli_dtype y_dtype,
                                      int64_t y_stride, int device, coli_stream stream) {
    REQUIRE(weights || T <= 0, "weights is NULL");
    REQUIRE(aligned4(weights), "weights must be 4-byte aligned");
    return gather_entry(pos, weights, T, K, Mat{rows, rows_dtype, n_rows, hidden, rows_stride}, base, base_stride,
                        Mat{y, y_dtype, T, hidden, y_stride}, device, (cudaStream_t)stream);
}

COLI_API coli_status coli_moe_combine_backward(const int32_t* pos, const float* weights, int T, int K, const void* dy,
                                               coli_dtype dy_dtype, int64_t dy_stride, int hidden, const void* rows,
                                               coli_dtype rows_dtype, int64_t rows_stride, int64_t n_rows, void* drows,
                                               int64_t drows_stride, float* dweights, int device, coli_stream stream) {
    const Mat mr{rows, rows_dtype, n_rows, hidden, rows_stride}, md{drows, rows_dtype, n_rows, hidden, drows_stride};
    const Mat mg{dy, dy_dtype, T, hidden, dy_stride};
    coli_status s = check_combine(pos, T, K, mr, dweights != nullptr, hidden);
    if (s != COLI_OK) return s;
    REQUIRE(dtype_ok(dy_dtype), "dy_dtype must be COLI_F32 or COLI_BF16");
    REQUIRE(device >= 0, "no such CUDA device");
    if (T == 0 || (!drows && !dweights)) return COLI_OK;
    TRY_ARG(check_mat(mg, "dy is NULL", "dy_stride is smaller than hidden", "dy is not aligned to its element"));
    REQUIRE(weights || !drows, "weights is NULL");
    REQUIRE(aligned4(weights) && aligned4(dweights), "weights and dweights must be 4-byte aligned");
    const size_t n = (size_t)T * K * 4;
    if (drows) {
        TRY_ARG(check_mat(md, "", "drows_stride is smaller than hidden", "drows is not aligned to its element"));
        REQUIRE(!dweights || same(md, mr) || !overlap(md, mr), "drows and rows overlap");
        REQUIRE(!overlap(md, mg), "drows and dy overlap");
        REQUIRE(!overlap(drows, md.bytes(), pos, n) && !overlap(drows, md.bytes(), weights, n), "drows overlaps an input");
    }
    if (dweights) {
        REQUIRE(!overlap(dweights, n, pos, n) && !overlap(dweights, n, weights, n) &&
                    !overlap(dweights, n, dy, mg.bytes()) && !overlap(dweights, n, rows, mr.bytes()),
                "dweights overlaps an input");
        REQUIRE(!drows || !overlap(dweights, n, drows, md.bytes()), "dweights and drows overlap");
    }
    DeviceGuard guard(device);
    REQUIRE(guard.ok, "no such CUDA device");
    cudaStream_t st = (cudaStream_t)stream;
    const Mat* d = drows ? &md : nullptr;
    using B = __nv_bfloat16;
    cudaError_t e;
    if (rows_dtype == COLI_F32)
        e = dy_dtype == COLI_F32 ? combine_backward<float, float>(pos, weights, T, K, mg, mr, d, dweights, st)
                                 : combine_backward<float, B>(pos, weights, T, K, mg, mr, d, dweights, st);
    else
        e = dy_dtype == COLI_F32 ? combine_backward<B, float>(pos, weights, T, K, mg, mr, d, dweights, st)
                                 : combine_backward<B, B>(pos, weights, T, K, mg, mr, d, dweights, st);
    return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "combine backward");
}

// route_backward.cu -- gradient of the router's weights, rows and input
// (coli_moe_route_backward).
#include "block.cuh"

#include <type_traits>

#define COLI_API extern "C" __attribute__((visibility("default")))

namespace coli {
namespace {

constexpr int kSms = 148;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// First index in [a, b) whose slot is >= bound (the list of an expert is
// ascending): eight parts at a time, so four rounds of loads for 2048 slots.
__device__ __forceinline__ int first_at_least(const int32_t* slot, int a, int b, int bound) {
    while (b - a > 8) {
        const int step = (b - a) >> 3;
        int below = 0;
#pragma unroll
        for (int j = 1; j < 8; ++j) below += slot[a + j * step - 1] < bound;
        const int a0 = a;
        a = a0 + below * step;
        if (below < 7) b = a0 + (below + 1) * step;
    }
    int below = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) below += a + j < b && slot[a + j] < bound;
    return a + below;
}

// What the sums need, once for all column slabs:
//  - dlogits[t][k] = w_k (dw_k - sum_j w_j dw_j): the weights are a softmax over
//    the selected logits, whose Jacobian is diag(w) - w w^T. One warp a token.
//  - inv: the plan's row of each slot;
//  - bound[c][e]: the first row of expert e whose token is >= c * chunk (of the
//    last c: its end).
// Blocks [0, n_tok) take tokens, [n_tok, n_tok + n_inv) rows, the others bounds.
struct Prep {
    const int32_t *ids, *offsets, *slot;
    const float *w, *dw;
    float* dl;
    int32_t *inv, *bound;
    int T, K, E, chunk, n_chunks, n_tok, n_inv;
};
__global__ void __launch_bounds__(256) route_prep_kernel(const Prep a) {
    const int lane = threadIdx.x & 31, n = a.T * a.K;
    if ((int)blockIdx.x < a.n_tok) {
        const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
        if (t < a.T) {
            float wk = 0.0f, gk = 0.0f;
            const size_t i = (size_t)t * a.K + lane;
            if (lane < a.K) {
                const int e = a.ids[i];
                wk = (unsigned)e < (unsigned)a.E ? a.w[i] : 0.0f;
                gk = wk != 0.0f ? a.dw[i] : 0.0f;  // an absent slot's dweights is not used
            }
            float m = wk * gk;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
            if (lane < a.K) a.dl[i] = wk != 0.0f ? wk * (gk - m) : 0.0f;
        }
    } else if ((int)blockIdx.x < a.n_tok + a.n_inv) {
        const int q = (blockIdx.x - a.n_tok) * 256 + threadIdx.x;
        if (q < n) {
            const int i = a.slot[q];
            if (i >= 0 && i < n) a.inv[i] = q;
        }
    } else {
        const int j = (blockIdx.x - a.n_tok - a.n_inv) * 256 + threadIdx.x;
        if (j < (a.n_chunks + 1) * a.E) {
            const int c = j / a.E, e = j % a.E;
            const int q0 = min(max(a.offsets[e], 0), n), q1 = min(max(a.offsets[e + 1], q0), n);
            const int t = min(c * a.chunk, a.T);
            a.bound[j] = t == 0 ? q0 : t == a.T ? q1 : first_at_least(a.slot, q0, q1, t * a.K);
        }
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
// the tokens; a warp takes four tokens at a time (K <= 8), a lane VC columns of each.
// The slots' rows and factors go through a buffer of the warp's, from which
// all lanes read two slots with one access. Most of its time are shared memory
// reads, 36 wavefronts a token and slab (13 of the 20 us there); gathering the
// rows from L2 took 45. A slot that is absent reads a row of zeros.
// ---------------------------------------------------------------------------
struct SlotRef {
    int row;  // its row's place in shared memory, in elements or bytes
    float d;
};

template <int VC>
struct Columns;
template <>
struct Columns<4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void add(float d, float2 (&acc)[2]) const {
        acc[0] = __ffma2_rn(make_float2(d, d), make_float2(v.x, v.y), acc[0]);
        acc[1] = __ffma2_rn(make_float2(d, d), make_float2(v.z, v.w), acc[1]);
    }
};
template <>
struct Columns<2> {
    float2 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
    __device__ __forceinline__ void add(float d, float2 (&acc)[1]) const { acc[0] = __ffma2_rn(make_float2(d, d), v, acc[0]); }
};
template <>
struct Columns<1> {
    float v;
    __device__ __forceinline__ void load(const float* p) { v = *p; }
    __device__ __forceinline__ void add(float d, float2 (&acc)[1]) const { acc[0].x = fmaf(d, v, acc[0].x); }
};

struct Dx {
    const int32_t* ids;
    const float *dl, *wr;
    int T, K, E, H, per, slabs, blocks;  // per: tokens of a block
    int vec;
    int64_t ldx;
};

template <typename XT, int VC>
__device__ __forceinline__ void route_dx_block(const Dx& a, XT* dx, int bx, int by, unsigned char* shared) {
    // [E + 1][32 * VC] columns of the router's rows, the last row zero; then each warp's two buffers of 32 slots
    float* slab = reinterpret_cast<float*>(shared);
    SlotRef* refs = reinterpret_cast<SlotRef*>(slab + (a.E + 1) * 32 * VC) + (threadIdx.x >> 5) * 64;
    const int32_t* ids = a.ids;
    const float *dl = a.dl, *wr = a.wr;
    const int T = a.T, K = a.K, E = a.E, H = a.H, per = a.per;
    const bool vec = a.vec;
    const int64_t ldx = a.ldx;
    constexpr int C = 32 * VC;
    const int c0 = bx * C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    // a warp's turn: its lanes hold the slots of G tokens, in groups of 8, 16 or 32 (zero rows behind the K-th)
    const int sh = K <= 8 ? 3 : K <= 16 ? 4 : 5, G = 32 >> sh, tg = lane >> sh, tk = lane & ((1 << sh) - 1);
    const int t1 = min(T, (by + 1) * per);
    int t = by * per + warp * G;
    auto fetch = [&](int at) {
        SlotRef r{E * C, 0.0f};
        if (tk < K && at + tg < t1) {
            const int i = (at + tg) * K + tk;
            const int id = ids[i];
            r.d = dl[i];
            if (r.d != 0.0f && (unsigned)id < (unsigned)E) r.row = id * C;
            else r.d = 0.0f;
        }
        return r;
    };
    SlotRef mine = fetch(t);
    cp_async_wait_all();
    __syncthreads();
    const float* col = slab + lane * VC;
    const int left = H - c0 - lane * VC;
    for (int flip = 0; t < t1; t += kWarps * G, flip ^= 1) {
        SlotRef* ref = refs + 32 * flip;
        ref[lane] = mine;
        __syncwarp();
        mine = fetch(t + kWarps * G);
        for (int g = 0; g < G && t + g < t1; ++g) {
            float2 sum[(VC + 1) / 2];
#pragma unroll
            for (int j = 0; j < (VC + 1) / 2; ++j) sum[j] = make_float2(0.0f, 0.0f);
            for (int k0 = 0; k0 < K; k0 += 8) {
                int4 r[4];  // two slots each
                Columns<VC> v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k] = reinterpret_cast<const int4*>(ref + (g << sh) + k0)[k];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[2 * k].load(col + r[k].x);
                    v[2 * k + 1].load(col + r[k].z);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[2 * k].add(__int_as_float(r[k].y), sum);
                    v[2 * k + 1].add(__int_as_float(r[k].w), sum);
                }
            }
            float acc[VC];
#pragma unroll
            for (int j = 0; j < VC; ++j) acc[j] = j & 1 ? sum[j / 2].y : sum[j / 2].x;
            XT* out = dx + (size_t)(t + g) * ldx + c0 + lane * VC;
            if (VC == 4 && vec) {
                if (left > 0) {
                    if constexpr (sizeof(XT) == 4) {
                        *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1 % VC], acc[2 % VC], acc[3 % VC]);
                    } else {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0], acc[1 % VC]),
                                             hi = __floats2bfloat162_rn(acc[2 % VC], acc[3 % VC]);
                        *reinterpret_cast<uint2*>(out) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < VC; ++j)
                    if (j < left) {
                        Raw<XT, 1> one;
                        const float f[1] = {acc[j]};
                        one.set(f);
                        one.store(out + j);
                    }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// drouter_w[e] and dbias[e]: sums over the expert's slots of dlogits * x[token].
// Again a token's row is needed K times, so a block keeps 256 bytes of columns
// of a chunk of tokens in shared memory, and beside them the chunk's slots in
// expert order (their places follow from the plan). A warp takes an expert and
// adds its rows in order, a lane 8 bytes of each. A block takes `per` chunks of
// its split one after another; its sums go to the split's part of the
// workspace, which route_sum_kernel adds in order; with one split they are the
// result. 22 us at 2048 x 8 x 6144 bf16, 256 experts. (A block per expert that
// walked its slots took 1200: the hottest expert has most tokens.) No unit is full:
// with dx, 56 % of the issue slots and 58 % of the shared memory pipe are in use,
// and warps wait for shared memory most; one block an SM has nothing to run while
// it fills its chunk or waits at its barriers.
// ---------------------------------------------------------------------------
constexpr int kRowBytes = 256;
constexpr int kRoom = 224 * 1024;        // shared memory of a chunk
constexpr int kMostShared = 226 * 1024;  // of any block: over all E and K, 229,364 bytes are the most
constexpr int kFirst = 6;           // slots a thread asks for at once (all of a chunk's, with K <= 8)

// Most tokens of a chunk: their rows, one zero row, their slots (an even number of each expert's), and two
// numbers an expert fit.
int chunk_of(int K, int E) { return (kRoom - kRowBytes - 16 * (E + 1)) / (kRowBytes + 8 * K); }

// Exclusive prefix sums of v[0..n) in place (n <= 1024), the total behind them.
__device__ __forceinline__ void prefix(int* v, int n, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = 2 * threadIdx.x;
    const int a = i < n ? v[i] : 0, b = i + 1 < n ? v[i + 1] : 0;
    int s = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int before = s - a - b;
    for (int w = 0; w < warp; ++w) before += sums[w];
    if (i < n) v[i] = before;
    if (i + 1 < n) v[i + 1] = before + a;
    if (threadIdx.x == kThreads - 1) v[n] = before + a + b;
    __syncthreads();
}

struct Rows {
    const int32_t *ids, *inv, *bound;
    const float* dl;
    int T, K, E, H, chunk, n_chunks, per, slabs;
    int64_t ldx;
    int vec, vec_out;
    float *part, *part_b;  // NULL: not wanted
};

template <typename XT>
__device__ __forceinline__ void route_rows_block(const Rows& a, const XT* x, int bx, int by, unsigned char* rows) {
    // rows [chunk + 1][256], the last one zero; slots [chunk * K + E]; place [E + 1] of an expert's first slot; first [E]
    __shared__ int next, sums[kWarps];
    constexpr int C = kRowBytes / sizeof(XT), V = 16 / sizeof(XT), P = 4 / sizeof(XT);  // P pairs of columns a lane
    const int K = a.K, E = a.E, H = a.H, chunk = a.chunk;
    SlotRef* refs = reinterpret_cast<SlotRef*>(rows + (chunk + 1) * kRowBytes);
    int* place = reinterpret_cast<int*>(refs + chunk * K + E);
    int* first = place + E + 1;
    const int c0 = bx * C, lane = threadIdx.x & 31;
    const SlotRef none{chunk * kRowBytes, 0.0f};  // the zero row: an absent slot
    if (threadIdx.x < kRowBytes / 4) reinterpret_cast<int*>(rows + chunk * kRowBytes)[threadIdx.x] = 0;
    grid_wait();
    const int k0 = by * a.per, k1 = min(a.n_chunks, k0 + a.per);
    for (int k = k0; k < k1; ++k) {
        const int t0 = k * chunk, t1 = min(a.T, t0 + chunk), ns = (t1 - t0) * K;
        for (int e = threadIdx.x; e < E; e += kThreads) {
            const int q0 = a.bound[k * E + e], q1 = a.bound[(k + 1) * E + e];
            first[e] = q0;
            place[e] = (min(max(q1 - q0, 0), ns) + 1) & ~1;  // even: two slots are read at a time
        }
        if (threadIdx.x == 0) next = 0;
        // the first slots' numbers are asked for ahead of the rows: behind them they came 8000 cycles later
        int e0[kFirst], i0[kFirst];
        float d0[kFirst];
#pragma unroll
        for (int j = 0; j < kFirst; ++j) {
            const int i = threadIdx.x + j * kThreads, at = t0 * K + i;
            e0[j] = i < ns ? a.ids[at] : -1;
            i0[j] = i < ns ? a.inv[at] : 0;
            d0[j] = i < ns ? a.dl[at] : 0.0f;
        }
        if (a.part) {
            if (a.vec) {
                for (int i = threadIdx.x; i < (t1 - t0) * 16; i += kThreads) {
                    const int t = i >> 4, c = (i & 15) * V;
                    if (c0 + c < H) cp_async16(smem_addr(rows) + i * 16, x + (size_t)(t0 + t) * a.ldx + c0 + c);
                }
            } else {
                for (int i = threadIdx.x; i < (t1 - t0) * C; i += kThreads) {
                    const int t = i / C, c = i % C;
                    if (c0 + c < H) reinterpret_cast<XT*>(rows)[i] = x[(size_t)(t0 + t) * a.ldx + c0 + c];
                }
            }
        }
        for (int i = threadIdx.x; i < ns + E; i += kThreads) refs[i] = none;
        __syncthreads();
        prefix(place, E, sums);
        // (offsets that are not a plan of these slots may list too many; even, as the places are)
        const int total = min(place[E], ns + E) & ~1;
        auto put = [&](int i, int e, int q, float d) {
            if (d == 0.0f || (unsigned)e >= (unsigned)E) return;
            const int p = place[e] + (q - first[e]);
            if (q >= first[e] && p >= 0 && p < place[e + 1] && p < total) refs[p] = SlotRef{i / K * kRowBytes, d};
        };
#pragma unroll
        for (int j = 0; j < kFirst; ++j) put(threadIdx.x + j * kThreads, e0[j], i0[j], d0[j]);
        for (int i = threadIdx.x + kFirst * kThreads; i < ns; i += kThreads)
            put(i, a.ids[t0 * K + i], a.inv[t0 * K + i], a.dl[t0 * K + i]);
        cp_async_wait_all();
        __syncthreads();
        for (;;) {
            int e = 0;
            if (lane == 0) e = atomicAdd(&next, 1);  // which warp takes an expert does not show in its sum
            e = __shfl_sync(0xffffffffu, e, 0);
            if (e >= E) break;
            const int q0 = min(place[e], total), q1 = min(place[e + 1], total);
            if (a.part) {
                float2 sum[P];
#pragma unroll
                for (int j = 0; j < P; ++j) sum[j] = make_float2(0.0f, 0.0f);
                const unsigned char* col = rows + lane * 8;
                auto add = [&](float f, const uint2& u) {
                    const float2 d = make_float2(f, f);
                    if constexpr (P == 1) {
                        sum[0] = __ffma2_rn(d, make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), sum[0]);
                    } else {
                        sum[0] = __ffma2_rn(d, make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u)), sum[0]);
                        sum[P - 1] = __ffma2_rn(d, make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)), sum[P - 1]);
                    }
                };
                auto group = [&](auto pairs, int q) {  // 2 * pairs slots from q on
                    constexpr int n = decltype(pairs)::value;
                    int4 r[n];
                    uint2 u[2 * n];
#pragma unroll
                    for (int s = 0; s < n; ++s) r[s] = reinterpret_cast<const int4*>(refs + q)[s];
#pragma unroll
                    for (int s = 0; s < n; ++s) {
                        u[2 * s] = *reinterpret_cast<const uint2*>(col + r[s].x);
                        u[2 * s + 1] = *reinterpret_cast<const uint2*>(col + r[s].z);
                    }
#pragma unroll
                    for (int s = 0; s < n; ++s) {
                        add(__int_as_float(r[s].y), u[2 * s]);
                        add(__int_as_float(r[s].w), u[2 * s + 1]);
                    }
                };
                int q = q0;
                for (; q + 8 <= q1; q += 8) group(std::integral_constant<int, 4>(), q);
                if (q + 4 <= q1) {
                    group(std::integral_constant<int, 2>(), q);
                    q += 4;
                }
                if (q < q1) group(std::integral_constant<int, 1>(), q);
                const int c = c0 + lane * 2 * P;
                float* out = a.part + ((size_t)by * E + e) * H + c;
                const bool more = k != k0;  // added to the sums of the chunks before
                if (c < H) {
                    if (a.vec_out) {
                        if constexpr (P == 2) {
                            float4 v = make_float4(sum[0].x, sum[0].y, sum[P - 1].x, sum[P - 1].y);
                            if (more) {
                                const float4 o = *reinterpret_cast<const float4*>(out);
                                v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
                            }
                            *reinterpret_cast<float4*>(out) = v;
                        } else {
                            float2 v = sum[0];
                            if (more) {
                                const float2 o = *reinterpret_cast<const float2*>(out);
                                v = make_float2(o.x + v.x, o.y + v.y);
                            }
                            *reinterpret_cast<float2*>(out) = v;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2 * P; ++j) {
                            const float v = j & 1 ? sum[j / 2].y : sum[j / 2].x;
                            if (c + j < H) out[j] = more ? out[j] + v : v;
                        }
                    }
                }
            }
            if (a.part_b && bx == 0) {
                float b = 0.0f;
                for (int q = q0 + lane; q < q1; q += 32) b += refs[q].d;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
                float* out = a.part_b + (size_t)by * E + e;
                if (lane == 0) *out = k != k0 ? *out + b : b;
            }
        }
        __syncthreads();
    }
}

// Both in one launch: they need the same preparation and nothing of one another,
// and a launch of its own costs each 2 us. The blocks of dx come first. (One
// block an SM: without the second bound the compiler saves registers for two.)
template <typename XT, int VC>
__global__ void __launch_bounds__(kThreads, 1) route_sums_kernel(const __grid_constant__ Dx d, const __grid_constant__ Rows r,
                                                                 const XT* x, XT* dx) {
    extern __shared__ __align__(16) unsigned char shared[];
    const int b = blockIdx.x;
    if (b < d.blocks) route_dx_block<XT, VC>(d, dx, b % d.slabs, b / d.slabs, shared);
    else route_rows_block<XT>(r, x, (b - d.blocks) % r.slabs, (b - d.blocks) / r.slabs, shared);
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

// How a call's tokens are cut: chunks of at most what a block's shared memory
// holds, `per` of them to a split, `splits` splits: as many as fill the GPU
// beside the column slabs, each of 128 tokens or more. The workspace's size
// depends on it, so it must not depend on the type: the fewer slabs, of bf16,
// count.
struct Cut {
    int chunk, n_chunks, per, splits;
};
int most_splits(int T, int H) {
    const int slabs = (H + 127) / 128;
    int n = kSms / slabs;
    if (n > (T + 127) / 128) n = (T + 127) / 128;
    return n < 1 ? 1 : n;
}
Cut cut_of(int T, int K, int E, int H) {
    const int n = most_splits(T, H);
    Cut c;
    const int share = T > 0 ? (T + n - 1) / n : 1, most = chunk_of(K, E);
    c.per = (share + most - 1) / most;
    c.chunk = (share + c.per - 1) / c.per;
    c.n_chunks = T > 0 ? (T + c.chunk - 1) / c.chunk : 1;
    c.splits = (c.n_chunks + c.per - 1) / c.per;
    return c;
}
// The workspace: parts of drouter_w and dbias (several splits), inv, bound.
struct Layout {
    int64_t part_b, inv, bound, total;  // in 4-byte words
};
Layout layout_of(const Cut& c, int T, int K, int E, int H) {
    auto up = [](int64_t n) { return (n + 3) / 4 * 4; };
    Layout l;
    l.part_b = c.splits > 1 ? up((int64_t)c.splits * E * H) : 0;
    l.inv = l.part_b + (c.splits > 1 ? up((int64_t)c.splits * E) : 0);
    l.bound = l.inv + up((int64_t)T * K);
    l.total = l.bound + up((int64_t)(c.n_chunks + 1) * E);
    return l;
}
// Words that hold the layout of so many tokens or fewer. Both numbers grow with T
// and are at least the cut's own (which may fall: 18945 tokens of 128 columns take
// 147 splits, 18944 take 148): splits <= n, and n_chunks <= n per
// <= n (ceil(T / n) / most + 1) <= (T + n) / most + n.
int64_t most_words(int T, int K, int E, int H) {
    const int n = most_splits(T, H);
    return layout_of(Cut{0, (T + n) / chunk_of(K, E) + n, 0, n}, T, K, E, H).total;
}

// Columns of a slab of all E router rows (and the zero row) in shared memory, in warps' widths.
int slab_columns(int E) {
    for (int vc : {4, 2}) if ((size_t)(E + 1) * 32 * vc * 4 <= 200 * 1024) return vc;
    return 1;
}

// dx (dx.p NULL: not wanted here) and the parts of drouter_w and dbias (NULL: not wanted).
template <typename XT>
cudaError_t route_sums(const Prep& p, const Mat& wr, const Mat& x, const Mat& dx, const Cut& c, float* dwr, float* dbias,
                       float* work, const Layout& l, cudaStream_t st) {
    constexpr int C = kRowBytes / sizeof(XT);
    const int T = p.T, K = p.K, E = p.E, H = x.cols;
    size_t smem = 0;
    const int vc = slab_columns(E);
    Dx d{p.ids, p.dl, (const float*)wr.p, T, K, E, H, 0, 1, 0, 0, dx.stride};
    if (dx.p) {
        d.slabs = (H + 32 * vc - 1) / (32 * vc);
        int n = kSms / d.slabs;
        if (n > (T + kWarps - 1) / kWarps) n = (T + kWarps - 1) / kWarps;
        if (n < 1) n = 1;
        d.per = (T + n - 1) / n;
        d.blocks = d.slabs * ((T + d.per - 1) / d.per);
        d.vec = H % 4 == 0 && wr.starts(16) && dx.starts(16);
        smem = (size_t)(E + 1) * 32 * vc * 4 + kWarps * 64 * sizeof(SlotRef);
    }
    Rows r{p.ids, p.inv, p.bound, p.dl, T, K, E, H, c.chunk, c.n_chunks, c.per, 1, x.stride};
    int blocks = d.blocks;
    if (dwr || dbias) {
        r.vec = x.starts(16) && H % (16 / sizeof(XT)) == 0;
        // one split writes the result itself, several their parts
        r.part = !dwr ? nullptr : c.splits > 1 ? work : dwr;
        r.part_b = !dbias ? nullptr : c.splits > 1 ? work + l.part_b : dbias;
        r.vec_out = H % 4 == 0 && ((uintptr_t)r.part & 15u) == 0;
        r.slabs = dwr ? (H + C - 1) / C : 1;
        blocks += r.slabs * c.splits;
        const size_t need = (size_t)(c.chunk + 1) * kRowBytes + ((size_t)c.chunk * K + E) * 8 + (size_t)(2 * E + 1) * 4;
        if (need > smem) smem = need;
    }
    if (blocks == 0) return cudaSuccess;
    auto k = vc == 4 ? route_sums_kernel<XT, 4> : vc == 2 ? route_sums_kernel<XT, 2> : route_sums_kernel<XT, 1>;
    cudaError_t e = allow_shared(k, kMostShared);
    if (e != cudaSuccess) return e;
    e = launch(k, blocks, kThreads, smem, st, true, d, r, (const XT*)x.p, (XT*)dx.p);
    if (e != cudaSuccess || c.splits == 1 || !(dwr || dbias)) return e;
    const int n = E * H;
    const bool v4 = H % 4 == 0 && (((uintptr_t)dwr | (uintptr_t)work) & 15u) == 0;
    const int V = v4 ? 4 : 1, sums = dwr ? (n / V + 255) / 256 : 1, need = (E + 255) / 256;
    return launch(v4 ? route_sum_kernel<4> : route_sum_kernel<1>, sums > need ? sums : need, 256, 0, st, true,
                  (const float*)r.part, c.splits, n, dwr, (const float*)r.part_b, E, dbias);
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
    return T > 0 ? most_words(T, K, E, H) * 4 : 0;
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
    const int64_t need = rows && T > 0 ? layout_of(cut_of(T, K, E, H), T, K, E, H).total * 4 : 0;
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
    const Cut c = cut_of(T, K, E, H);
    const Layout l = layout_of(c, T, K, E, H);
    Prep p{};
    p.ids = ids, p.offsets = offsets, p.slot = slot, p.w = weights, p.dw = dweights, p.dl = dlogits;
    p.T = T, p.K = K, p.E = E, p.chunk = c.chunk, p.n_chunks = c.n_chunks;
    p.n_tok = (T + 7) / 8;
    if (rows) {
        p.inv = (int32_t*)work + l.inv;
        p.bound = (int32_t*)work + l.bound;
        p.n_inv = (int)(((int64_t)T * K + 255) / 256);
    }
    const int n_bound = rows ? ((c.n_chunks + 1) * E + 255) / 256 : 0;
    e = launch(route_prep_kernel, p.n_tok + p.n_inv + n_bound, 256, 0, st, false, p);
    if (e != cudaSuccess) return block_cuda_fail(e, "route backward: logits");
    // few slots read fewer router rows than a slab of all of them holds
    const bool gather = dx && (int64_t)T * K < E;
    if (gather) {
        e = launch_gather_sum(ids, dlogits, true, T, K, mw, nullptr, mdx, st, true);
        if (e != cudaSuccess) return block_cuda_fail(e, "route backward: dx");
    }
    const Mat to{gather ? nullptr : dx, dtype, T, H, dx_stride};
    e = dtype == COLI_F32 ? route_sums<float>(p, mw, mx, to, c, drouter_w, dbias, (float*)work, l, st)
                          : route_sums<__nv_bfloat16>(p, mw, mx, to, c, drouter_w, dbias, (float*)work, l, st);
    if (e != cudaSuccess) return block_cuda_fail(e, "route backward: sums");
    return COLI_OK;
}

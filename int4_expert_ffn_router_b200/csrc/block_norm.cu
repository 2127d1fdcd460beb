// block_norm.cu -- the norms around a block with its gate and scales
// (coli_block_norm) and their gradients.
#include "block.cuh"

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
    float *part;            // [grid][3][H] partial sums of dpre, dpost, dgate
    int want;               // bit 0: dpre, bit 1: dpost, bit 2: dgate
};

// A sum of squares that fp32 holds well: it neither overflowed nor lost to
// underflow anything that eps does not hide (a square below 2^-126 is lost).
__device__ __forceinline__ bool sum_ok(float ss, float eps) { return ss <= 3e37f && (ss >= 1e-24f || eps >= 1e-12f); }
__device__ __forceinline__ float rms_scale(float ss, int H, float eps) { return rsqrtf(ss / (float)H + eps); }
__device__ __forceinline__ float rms_scale(double ss, int H, float eps) { return (float)(1.0 / sqrt(ss / H + (double)eps)); }

template <int V>
__device__ __forceinline__ void load_gain(const float* g, int c, float (&v)[V]) {
    if (!g) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 1.0f;
    } else if constexpr (V == 8) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(g + c)), b = __ldg(reinterpret_cast<const float4*>(g + c) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = __ldg(g + c);
    }
}

// ---------------------------------------------------------------------------
// Forward, one block a row. A thread's N x V columns of x and y stay in
// registers between the two sums.
// ---------------------------------------------------------------------------
template <typename XT, typename YT, typename NT, int V, int N>
__global__ void __launch_bounds__(1024) block_norm_kernel(NormArgs a) {
    __shared__ float red[2][32];
    __shared__ double red64[2][32];
    const int t = blockIdx.x, H = a.H;
    const XT* x = (const XT*)a.x + (size_t)t * a.ldx;
    const YT* y = (const YT*)a.y + (size_t)t * a.ldy;
    float s[N * V];
    Raw<XT, V> rx[N];
    Raw<YT, V> ry[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        rx[i].zero();
        ry[i].zero();
        if (c < H) {
            rx[i].load(x + c);
            if (a.has_prev) ry[i].load(y + c);
        }
    }
    float scale = 1.0f;
    if (a.has_prev) {
        scale = a.ys * (a.token ? a.token[t] : 1.0f);
        float rho = 1.0f;
        if (a.post_norm) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float v[V];
                ry[i].get(v);
#pragma unroll
                for (int j = 0; j < V; ++j) ss[0] = fmaf(v[j], v[j], ss[0]);
            }
            block_sum<float, 1>(ss, red[0]);
            rho = rms_scale(ss[0], H, a.eps_post);
            if (!sum_ok(ss[0], a.eps_post)) {
                double dd[1] = {0.0};
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float v[V];
                    ry[i].get(v);
#pragma unroll
                    for (int j = 0; j < V; ++j) dd[0] += (double)v[j] * v[j];
                }
                block_sum<double, 1>(dd, red64[0]);
                rho = rms_scale(dd[0], H, a.eps_post);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= H) {
#pragma unroll
                for (int j = 0; j < V; ++j) s[i * V + j] = 0.0f;
                continue;
            }
            float vx[V], vy[V], p[V], g[V];
            rx[i].get(vx);
            ry[i].get(vy);
            load_gain<V>(a.post, c, p);
            load_gain<V>(a.gate, c, g);
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = fmaf(scale * g[j], vy[j] * rho * p[j], a.xs * vx[j]);
            rx[i].set(o);
            rx[i].store((XT*)a.xo + (size_t)t * a.ldxo + c);
            rx[i].get(vx);  // as stored: what a later read of x_out sees
#pragma unroll
            for (int j = 0; j < V; ++j) s[i * V + j] = vx[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[V];
            rx[i].get(v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[i * V + j] = v[j];
        }
    }
    if (!a.has_next) return;
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < N * V; ++i) ss[0] = fmaf(s[i], s[i], ss[0]);
    block_sum<float, 1>(ss, red[1]);
    float r = rms_scale(ss[0], H, a.eps_pre);
    if (!sum_ok(ss[0], a.eps_pre)) {
        double dd[1] = {0.0};
#pragma unroll
        for (int i = 0; i < N * V; ++i) dd[0] += (double)s[i] * s[i];
        block_sum<double, 1>(dd, red64[1]);
        r = rms_scale(dd[0], H, a.eps_pre);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= H) continue;
        float q[V], o[V];
        load_gain<V>(a.pre, c, q);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = s[i * V + j] * r * q[j];
        Raw<NT, V> out;
        out.set(o);
        out.store((NT*)a.n + (size_t)t * a.ldn + c);
    }
}

// Rows too wide for registers: the same sums over columns that a thread reads
// again from memory (x_out again after it stored it, by the same thread).
template <typename XT, typename YT, typename NT>
__global__ void __launch_bounds__(1024) block_norm_wide_kernel(NormArgs a) {
    __shared__ float red[2][32];
    __shared__ double red64[2][32];
    const int t = blockIdx.x, H = a.H;
    const XT* x = (const XT*)a.x + (size_t)t * a.ldx;
    const YT* y = (const YT*)a.y + (size_t)t * a.ldy;
    XT* xo = a.has_prev ? (XT*)a.xo + (size_t)t * a.ldxo : nullptr;
    float ss[1] = {0.0f};
    if (a.has_prev) {
        float rho = 1.0f;
        if (a.post_norm) {
            for (int c = threadIdx.x; c < H; c += blockDim.x) {
                Raw<YT, 1> r;
                r.load(y + c);
                float v[1];
                r.get(v);
                ss[0] = fmaf(v[0], v[0], ss[0]);
            }
            block_sum<float, 1>(ss, red[0]);
            rho = rms_scale(ss[0], H, a.eps_post);
            if (!sum_ok(ss[0], a.eps_post)) {
                double dd[1] = {0.0};
                for (int c = threadIdx.x; c < H; c += blockDim.x) {
                    Raw<YT, 1> r;
                    r.load(y + c);
                    float v[1];
                    r.get(v);
                    dd[0] += (double)v[0] * v[0];
                }
                block_sum<double, 1>(dd, red64[0]);
                rho = rms_scale(dd[0], H, a.eps_post);
            }
        }
        const float scale = a.ys * (a.token ? a.token[t] : 1.0f);
        ss[0] = 0.0f;
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            Raw<XT, 1> rx;
            Raw<YT, 1> ry;
            rx.load(x + c);
            ry.load(y + c);
            float vx[1], vy[1], p[1], g[1];
            rx.get(vx);
            ry.get(vy);
            load_gain<1>(a.post, c, p);
            load_gain<1>(a.gate, c, g);
            vx[0] = fmaf(scale * g[0], vy[0] * rho * p[0], a.xs * vx[0]);
            rx.set(vx);
            rx.store(xo + c);
            rx.get(vx);
            ss[0] = fmaf(vx[0], vx[0], ss[0]);
        }
        x = xo;
    } else {
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            Raw<XT, 1> rx;
            rx.load(x + c);
            float v[1];
            rx.get(v);
            ss[0] = fmaf(v[0], v[0], ss[0]);
        }
    }
    if (!a.has_next) return;
    block_sum<float, 1>(ss, red[1]);
    float r = rms_scale(ss[0], H, a.eps_pre);
    if (!sum_ok(ss[0], a.eps_pre)) {
        double dd[1] = {0.0};
        for (int c = threadIdx.x; c < H; c += blockDim.x) {
            Raw<XT, 1> rx;
            rx.load(x + c);
            float v[1];
            rx.get(v);
            dd[0] += (double)v[0] * v[0];
        }
        block_sum<double, 1>(dd, red64[1]);
        r = rms_scale(dd[0], H, a.eps_pre);
    }
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
        Raw<XT, 1> rx;
        rx.load(x + c);
        float v[1], q[1];
        rx.get(v);
        load_gain<1>(a.pre, c, q);
        v[0] = v[0] * r * q[0];
        Raw<NT, 1> out;
        out.set(v);
        out.store((NT*)a.n + (size_t)t * a.ldn + c);
    }
}

// ---------------------------------------------------------------------------
// Backward. With sh = s r and yh = y rho (the normalised rows):
//   ds = dxo + r (q dn - sh mean(sh q dn))      dx = xs ds      dq = sum_t sh dn
//   dz = ys u g ds (z = yh p)                   dg = sum_t ys u z ds, du = sum_c ys g z ds
//   dy = rho (p dz - yh mean(yh p dz))          dp = sum_t yh dz
// Two rounds of sums a row: {s^2, s q dn, y^2}, then {y p dz, ys g z ds}. A block
// takes the rows b, b + grid, ... and keeps the sums over its rows of its
// threads' columns (dq, dp, dg) in registers; sum_parts_kernel adds the blocks'.
// ---------------------------------------------------------------------------
template <typename XT, typename YT, typename NT, int V, int N>
__global__ void __launch_bounds__(1024) block_norm_backward_kernel(NormArgs a) {
    __shared__ float red[2][32 * 3];
    __shared__ double red64[2][32 * 3];
    const int H = a.H;
    float dq[N * V], dp[N * V], dg[N * V];
#pragma unroll
    for (int i = 0; i < N * V; ++i) dq[i] = dp[i] = dg[i] = 0.0f;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        Raw<XT, V> rs[N], ro[N];
        Raw<YT, V> ry[N];
        Raw<NT, V> rn[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            rs[i].zero();
            ro[i].zero();
            ry[i].zero();
            rn[i].zero();
            if (c < H) {
                rs[i].load((const XT*)a.x + (size_t)t * a.ldx + c);
                if (a.has_prev) ry[i].load((const YT*)a.y + (size_t)t * a.ldy + c);
                if (a.dxo) ro[i].load((const XT*)a.dxo + (size_t)t * a.lddxo + c);
                if (a.has_next) rn[i].load((const NT*)a.dn + (size_t)t * a.lddn + c);
            }
        }
        const float u = a.token ? a.token[t] : 1.0f;
        float r = 0.0f, m1 = 0.0f, rho = 1.0f;
        {
            float v[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (i * blockDim.x + threadIdx.x) * V;
                if (c >= H) continue;
                float s[V], n[V], y[V], q[V];
                rs[i].get(s);
                rn[i].get(n);
                ry[i].get(y);
                load_gain<V>(a.pre, c, q);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[0] = fmaf(s[j], s[j], v[0]);
                    v[1] = fmaf(s[j], q[j] * n[j], v[1]);
                    v[2] = fmaf(y[j], y[j], v[2]);
                }
            }
            block_sum<float, 3>(v, red[0]);
            const bool ok = (!a.has_next || sum_ok(v[0], a.eps_pre)) && (!a.post_norm || sum_ok(v[2], a.eps_post));
            if (ok) {
                r = rms_scale(v[0], H, a.eps_pre);
                m1 = v[1] * r / (float)H;
                if (a.post_norm) rho = rms_scale(v[2], H, a.eps_post);
            } else {
                double w[3] = {0.0, 0.0, 0.0};
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int c = (i * blockDim.x + threadIdx.x) * V;
                    if (c >= H) continue;
                    float s[V], n[V], y[V], q[V];
                    rs[i].get(s);
                    rn[i].get(n);
                    ry[i].get(y);
                    load_gain<V>(a.pre, c, q);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        w[0] += (double)s[j] * s[j];
                        w[1] += (double)s[j] * q[j] * n[j];
                        w[2] += (double)y[j] * y[j];
                    }
                }
                block_sum<double, 3>(w, red64[0]);
                r = rms_scale(w[0], H, a.eps_pre);
                m1 = (float)(w[1] * (double)r / H);
                if (a.post_norm) rho = rms_scale(w[2], H, a.eps_post);
            }
        }
        float ds[N * V];
        float v[2] = {0.0f, 0.0f};  // sum of yh p dz, of ys g z ds
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= H) continue;
            float s[V], n[V], y[V], o[V], q[V], p[V], g[V];
            ro[i].get(o);
            if (a.has_next) {
                rs[i].get(s);
                rn[i].get(n);
                load_gain<V>(a.pre, c, q);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float sh = s[j] * r;
                    dq[i * V + j] = fmaf(sh, n[j], dq[i * V + j]);
                    o[j] = fmaf(r, fmaf(-sh, m1, q[j] * n[j]), o[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) ds[i * V + j] = o[j];
            if (a.has_prev) {
                ry[i].get(y);
                load_gain<V>(a.post, c, p);
                load_gain<V>(a.gate, c, g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float yh = y[j] * rho, zd = a.ys * yh * p[j] * o[j], dz = a.ys * u * g[j] * o[j];
                    dp[i * V + j] = fmaf(yh, dz, dp[i * V + j]);
                    dg[i * V + j] = fmaf(u, zd, dg[i * V + j]);
                    v[0] = fmaf(yh, p[j] * dz, v[0]);
                    v[1] = fmaf(g[j], zd, v[1]);
                    o[j] *= a.xs;
                }
            }
            if (a.dx) {
                Raw<XT, V> out;
                out.set(o);
                out.store((XT*)a.dx + (size_t)t * a.lddx + c);
            }
        }
        if (!a.has_prev) {
            __syncthreads();  // the next row's sums reuse red[0]
            continue;
        }
        block_sum<float, 2>(v, red[1]);
        if (a.dtoken && threadIdx.x == 0) a.dtoken[t] = v[1];
        if (!a.dy) continue;
        const float m2 = a.post_norm ? v[0] / (float)H : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * blockDim.x + threadIdx.x) * V;
            if (c >= H) continue;
            float y[V], p[V], g[V];
            ry[i].get(y);
            load_gain<V>(a.post, c, p);
            load_gain<V>(a.gate, c, g);
#pragma unroll
            for (int j = 0; j < V; ++j)
                y[j] = rho * fmaf(-(y[j] * rho), m2, p[j] * (a.ys * u * g[j] * ds[i * V + j]));
            Raw<YT, V> out;
            out.set(y);
            out.store((YT*)a.dy + (size_t)t * a.lddy + c);
        }
    }
    if (!a.want) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= H) continue;
        float* out = a.part + (size_t)blockIdx.x * 3 * H + c;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (a.want & 1) out[j] = dq[i * V + j];
            if (a.want & 2) out[(size_t)H + j] = dp[i * V + j];
            if (a.want & 4) out[(size_t)2 * H + j] = dg[i * V + j];
        }
    }
}

// Rows too wide for registers: the columns are read again in each round, and
// the sums over a block's rows grow in its part of the workspace.
template <typename XT, typename YT, typename NT>
__global__ void __launch_bounds__(1024) block_norm_backward_wide_kernel(NormArgs a) {
    __shared__ double red64[2][32 * 3];
    const int H = a.H;
    float* part = a.want ? a.part + (size_t)blockIdx.x * 3 * H : nullptr;
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
            float s, y, n, o, q[1];
            row(c, s, y, n, o);
            load_gain<1>(a.pre, c, q);
            w[0] += (double)s * s;
            w[1] += (double)s * q[0] * n;
            w[2] += (double)y * y;
        }
        block_sum<double, 3>(w, red64[0]);
        const float r = rms_scale(w[0], H, a.eps_pre);
        const float m1 = (float)(w[1] * (double)r / H);
        const float rho = a.post_norm ? rms_scale(w[2], H, a.eps_post) : 1.0f;
        double v[2] = {0.0, 0.0};
        float m2 = 0.0f;
        for (int round = 0; round < 2; ++round) {
            for (int c = threadIdx.x; c < H; c += blockDim.x) {
                float s, y, n, o, q[1], p[1], g[1];
                row(c, s, y, n, o);
                load_gain<1>(a.pre, c, q);
                load_gain<1>(a.post, c, p);
                load_gain<1>(a.gate, c, g);
                const float sh = s * r;
                if (a.has_next) o = fmaf(r, fmaf(-sh, m1, q[0] * n), o);
                const float yh = y * rho, zd = a.ys * yh * p[0] * o, dz = a.ys * u * g[0] * o;
                if (round == 0) {
                    v[0] += (double)yh * p[0] * dz;
                    v[1] += (double)g[0] * zd;
                    if (a.want & 1) part[c] = first ? sh * n : fmaf(sh, n, part[c]);
                    if (a.want & 2) part[H + c] = first ? yh * dz : fmaf(yh, dz, part[H + c]);
                    if (a.want & 4) part[2 * H + c] = first ? u * zd : fmaf(u, zd, part[2 * H + c]);
                } else {  // every input of this column has been read: dx and dy may be inputs
                    float f[1] = {a.has_prev ? a.xs * o : o};
                    if (a.dx) {
                        Raw<XT, 1> out;
                        out.set(f);
                        out.store((XT*)a.dx + (size_t)t * a.lddx + c);
                    }
                    if (a.dy) {
                        f[0] = rho * fmaf(-yh, m2, p[0] * dz);
                        Raw<YT, 1> out;
                        out.set(f);
                        out.store((YT*)a.dy + (size_t)t * a.lddy + c);
                    }
                }
            }
            if (round == 0) {
                block_sum<double, 2>(v, red64[1]);
                if (a.dtoken && threadIdx.x == 0) a.dtoken[t] = (float)v[1];
                m2 = a.post_norm ? (float)(v[0] / H) : 0.0f;
            }
        }
    }
}

// out[k][c] = sum over the blocks of part[b][k][c], in block order: 32 columns
// and 8 runs of blocks a block.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* part, int n, int H, float* o0, float* o1, float* o2) {
    __shared__ float sh[8][32];
    grid_wait();
    const int which = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float* out = which == 0 ? o0 : which == 1 ? o1 : o2;
    if (!out) return;
    const int per = (n + 7) / 8, b0 = g * per, b1 = min(n, b0 + per);
    float acc = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int b = b0; b < b1; ++b) acc += part[((size_t)b * 3 + which) * H + c];
    sh[g][threadIdx.x & 31] = acc;
    __syncthreads();
    if (g == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) acc += sh[i][threadIdx.x];
        out[c] = acc;
    }
}

constexpr int kPartBlocks = 296;  // blocks whose partial sums the workspace holds
int backward_grid(int T) { return T < kPartBlocks ? T : kPartBlocks; }

// V, N and threads for rows of H columns: 8-column accesses in up to 1024
// threads; single columns otherwise; N == 0: too wide for registers.
struct Shape {
    int V, N, threads;
};
Shape shape_of(int H, bool vec) {
    const int V = vec ? 8 : 1;
    const int n = (H + V - 1) / V;
    for (int N : {1, 2, 8}) {
        if (vec && N > 2) break;
        const int th = ((n + N - 1) / N + 31) / 32 * 32;
        if (th <= (vec ? 1024 : 512) || (!vec && N == 8 && th <= 1024)) return {V, N, th};
    }
    return {V, 0, 1024};
}

using B = __nv_bfloat16;

template <typename XT, typename YT, typename NT>
cudaError_t forward_typed(const NormArgs& a, bool vec, cudaStream_t st) {
    const Shape s = shape_of(a.H, vec);
    void (*k)(NormArgs) = s.N == 0   ? block_norm_wide_kernel<XT, YT, NT>
                          : s.V == 8 ? (s.N == 1 ? block_norm_kernel<XT, YT, NT, 8, 1> : block_norm_kernel<XT, YT, NT, 8, 2>)
                          : s.N == 1 ? block_norm_kernel<XT, YT, NT, 1, 1>
                          : s.N == 2 ? block_norm_kernel<XT, YT, NT, 1, 2>
                                     : block_norm_kernel<XT, YT, NT, 1, 8>;
    return launch(k, a.T, s.threads, 0, st, false, a);
}

template <typename XT, typename YT, typename NT>
cudaError_t backward_typed(const NormArgs& a, bool vec, cudaStream_t st) {
    const Shape s = shape_of(a.H, vec);
    void (*k)(NormArgs) = s.N == 0 ? block_norm_backward_wide_kernel<XT, YT, NT>
                          : s.V == 8
                              ? (s.N == 1 ? block_norm_backward_kernel<XT, YT, NT, 8, 1> : block_norm_backward_kernel<XT, YT, NT, 8, 2>)
                          : s.N == 1 ? block_norm_backward_kernel<XT, YT, NT, 1, 1>
                          : s.N == 2 ? block_norm_backward_kernel<XT, YT, NT, 1, 2>
                                     : block_norm_backward_kernel<XT, YT, NT, 1, 8>;
    return launch(k, backward_grid(a.T), s.threads, 0, st, false, a);
}

template <bool fwd>
cudaError_t by_type(const NormArgs& a, coli_dtype xt, coli_dtype yt, coli_dtype nt, bool vec, cudaStream_t st) {
    auto go = [&](auto x, auto y, auto n) {
        if constexpr (fwd) return forward_typed<decltype(x), decltype(y), decltype(n)>(a, vec, st);
        else return backward_typed<decltype(x), decltype(y), decltype(n)>(a, vec, st);
    };
    auto with_n = [&](auto x, auto y) { return nt == COLI_F32 ? go(x, y, float()) : go(x, y, B()); };
    auto with_y = [&](auto x) { return yt == COLI_F32 ? with_n(x, float()) : with_n(x, B()); };
    return xt == COLI_F32 ? with_y(float()) : with_y(B());
}

bool gain_vec(const float* p) { return ((uintptr_t)p & 15u) == 0; }

#define REQUIRE(cond, msg)                                \
    do {                                                  \
        if (!(cond)) return block_fail(COLI_EINVAL, msg); \
    } while (0)

void set_params(NormArgs& a, const coli_block_params* prev, const coli_block_params* next) {
    a.has_prev = prev != nullptr;
    a.has_next = next != nullptr;
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
    bool vec = H % 8 == 0 && x->vec() && gain_vec(a.pre) && gain_vec(a.post) && gain_vec(a.gate);
    if (prev) {
        a.y = y->p;
        a.ldy = y->stride;
        a.xo = x_out->p ? const_cast<void*>(x_out->p) : nullptr;
        a.ldxo = x_out->stride;
        vec = vec && y->vec() && x_out->vec();
    }
    if (next) {
        a.n = const_cast<void*>(n->p);
        a.ldn = n->stride;
        vec = vec && n->vec();
    }
    const cudaError_t e = by_type<true>(a, x->t, prev ? y->t : x->t, next ? n->t : x->t, vec, st);
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
    return (int64_t)backward_grid(T) * 3 * H * 4;
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
    const int want = (dpre_gain ? 1 : 0) | (dpost_gain ? 2 : 0) | (dgate ? 4 : 0);
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
    a.part = (float*)work;
    a.want = want;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        const bool vec = H % 8 == 0 && ms.vec() && (!prev || my.vec()) && (!next || mn.vec()) && (!dx_out || mo.vec()) &&
                         (!dx || mdx.vec()) && (!dy || mdy.vec()) && gain_vec(a.pre) && gain_vec(a.post) && gain_vec(a.gate);
        e = by_type<false>(a, x_dtype, prev ? y_dtype : x_dtype, next ? n_dtype : x_dtype, vec, s);
        if (e != cudaSuccess) return block_cuda_fail(e, "block norm backward");
    }
    if (!want) return COLI_OK;
    e = launch(sum_parts_kernel, dim3((H + 31) / 32, 3), 256, 0, s, false, (const float*)work, backward_grid(T), H,
               dpre_gain, dpost_gain, dgate);
    return e == cudaSuccess ? COLI_OK : block_cuda_fail(e, "block norm backward: gains");
}

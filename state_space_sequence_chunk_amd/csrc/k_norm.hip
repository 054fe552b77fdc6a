// Group norm with an activation, channels last, and its gradients.
//
// For each token and group of n channels (mean m only where it is taken):
//     u = x, or x silu(z) (gate before);   nh = (u - m) r,  r = (mean (u - m)^2 + eps)^-1/2
//     o = nh w + b;   out = o, silu(o), or o silu(z) (gate after)
// and backwards, with dO the gradient arriving at o and dn = dO w:
//     dw = sum dO nh,  db = sum dO,  du = r (dn - [mean dn] - nh mean(dn nh))
//
// Bound by memory: every input is read once and every output written once. tpg threads (a
// power of two) hold one group of one token in registers, in vectors of 8 or 4 channels where n
// allows it and else one by one; statistics are fp32 sums over registers,
// then a butterfly, then LDS where a group takes more than one wave. The mean is taken first
// and the squares of the differences after it, from the registers.
//
// 32768 x 5120 bf16 channels with a gate, 1.0 GB: 181 us, 5.6 TB/s; two rows of 5120: 4.2 us; backwards
// 16384 x 5120 with bf16 x and z, 1.3 GB: 283 us with its parameters, 4.7 TB/s.
//
// Backwards a thread keeps its channels over all the tokens it takes and adds up dw and db
// for them in registers; the rows of partial sums are added in a fixed order by a second
// kernel, so equal calls give equal bits.
#include <algorithm>
#include <type_traits>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp2_fast(-kLog2e * x)); }

// V values (8, 4 or 1) as one or two accesses of up to 16 bytes.
template <int V, typename T> __device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = to_f32(p[0]);
    } else if constexpr (sizeof(T) == 2) {
        typedef bf16 vec __attribute__((ext_vector_type(V)));
        const vec x = *(const vec*)p;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)x[i];
    } else {
#pragma unroll
        for (int h = 0; h < V; h += 4) {
            const f32x4 x = *(const f32x4*)(p + h);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h + i] = x[i];
        }
    }
}
template <int V, typename T> __device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        p[0] = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 2) {
        typedef bf16 vec __attribute__((ext_vector_type(V)));
        vec x;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (bf16)v[i];
        *(vec*)p = x;
    } else {
#pragma unroll
        for (int h = 0; h < V; h += 4) *(f32x4*)(p + h) = f32x4{v[h], v[h + 1], v[h + 2], v[h + 3]};
    }
}

// Sum over the tpg threads of a group; `part` has a float for every wave of the workgroup.
// Every thread of the workgroup calls it.
__device__ __forceinline__ float group_sum(float v, int tpg, float* part) {
    const int width = tpg < 64 ? tpg : 64;
    for (int o = 1; o < width; o <<= 1) v += __shfl_xor(v, o);
    if (tpg > 64) {
        const int w = threadIdx.x >> 6, nw = tpg >> 6, w0 = w / nw * nw;
        __syncthreads();  // the last sum's readers are done
        if ((threadIdx.x & 63) == 0) part[w] = v;
        __syncthreads();
        v = 0.f;
        for (int i = 0; i < nw; ++i) v += part[w0 + i];
    }
    return v;
}

// u of this thread's channels, normalised in place: u <- nh; returns r.
template <int V, int K>
__device__ __forceinline__ float normalise(float (&u)[K][V], const bool (&in)[K], int n, int tpg, bool center,
                                           float eps, float* part) {
    float s = 0.f;
    if (center) {
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) s += u[j][i];
        const float m = group_sum(s, tpg, part) / (float)n;
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) u[j][i] = in[j] ? u[j][i] - m : 0.f;
        s = 0.f;
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s += u[j][i] * u[j][i];
    const float r = 1.f / sqrtf(group_sum(s, tpg, part) / (float)n + eps);
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) u[j][i] *= r;
    return r;
}

template <typename TX, typename TZ, typename TO, int V, int K, int NTHR>
__global__ __launch_bounds__(NTHR) void group_norm_kernel(const TX* __restrict__ x, const TZ* __restrict__ z,
                                                          const float* __restrict__ wt,
                                                          const float* __restrict__ bs, TO* __restrict__ out,
                                                          long slots, int groups, int n, int tpg, int act,
                                                          int center, float eps) {
    __shared__ float part[16];
    const long slot = (long)blockIdx.x * (blockDim.x / tpg) + threadIdx.x / tpg;
    const bool live = slot < slots;
    const int lane = threadIdx.x & (tpg - 1), grp = (int)((live ? slot : 0) % groups);
    const size_t base = (size_t)(live ? slot : 0) * n;
    float u[K][V], zv[K][V];
    bool in[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int e = (j * tpg + lane) * V;
        in[j] = live && e < n;
        if (in[j]) {
            load_vec<V>(x + base + e, u[j]);
            if (act >= kActGatePre) load_vec<V>(z + base + e, zv[j]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) u[j][i] = zv[j][i] = 0.f;
        }
        if (act == kActGatePre) {
#pragma unroll
            for (int i = 0; i < V; ++i) u[j][i] *= zv[j][i] * sigmoid(zv[j][i]);
        }
    }
    normalise<V, K>(u, in, n, tpg, center != 0, eps, part);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int e = (j * tpg + lane) * V;
        if (in[j]) {
            float o[V], w[V], b[V];
            if (wt) load_vec<V>(wt + (size_t)grp * n + e, w);
            if (bs) load_vec<V>(bs + (size_t)grp * n + e, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = u[j][i] * (wt ? w[i] : 1.f) + (bs ? b[i] : 0.f);
                if (act == kActSilu) o[i] *= sigmoid(o[i]);
                if (act == kActGatePost) o[i] *= zv[j][i] * sigmoid(zv[j][i]);
            }
            store_vec<V>(out + base + e, o);
        }
    }
}

template <typename TX, typename TZ, int V, int K, int NTHR>
__global__ __launch_bounds__(NTHR) void group_norm_backward_kernel(
    const TX* __restrict__ x, const TZ* __restrict__ z, const float* __restrict__ wt,
    const float* __restrict__ bs, const float* __restrict__ dy, float* __restrict__ dx,
    float* __restrict__ dz, float* __restrict__ dwp, float* __restrict__ dbp, long tokens, int groups, int n,
    int tpg, int act, int center, float eps, int gpw, int tpw, int tblocks) {
    __shared__ float part[16];
    const int slot = threadIdx.x / tpg, lane = threadIdx.x & (tpg - 1);
    const int grp = blockIdx.x * gpw + slot % gpw, row = blockIdx.y * tpw + slot / gpw;
    const bool mine = slot < gpw * tpw && grp < groups;
    const int C = groups * n, c0 = (mine ? grp : 0) * n;
    float w[K][V], b[K][V], dw[K][V], db[K][V];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int e = (j * tpg + lane) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[j][i] = 1.f;
            b[j][i] = dw[j][i] = db[j][i] = 0.f;
        }
        if (mine && e < n) {
            if (wt) load_vec<V>(wt + c0 + e, w[j]);
            if (bs) load_vec<V>(bs + c0 + e, b[j]);
        }
    }
    // every thread of the workgroup makes the same number of turns (the sums wait for all)
    for (long t0 = 0; t0 < tokens; t0 += (long)tblocks * tpw) {
        const long t = t0 + row;
        const bool live = mine && t < tokens;
        const size_t base = (size_t)(live ? t : 0) * C + c0;
        float u[K][V], xv[K][V], zv[K][V], d[K][V];
        bool in[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int e = (j * tpg + lane) * V;
            in[j] = live && e < n;
            if (in[j]) {
                load_vec<V>(x + base + e, xv[j]);
                load_vec<V>(dy + base + e, d[j]);
                if (act >= kActGatePre) load_vec<V>(z + base + e, zv[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) xv[j][i] = zv[j][i] = d[j][i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                u[j][i] = act == kActGatePre ? xv[j][i] * zv[j][i] * sigmoid(zv[j][i]) : xv[j][i];
        }
        const float r = normalise<V, K>(u, in, n, tpg, center != 0, eps, part);
        float sn = 0.f, snh = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float gz[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float o = u[j][i] * w[j][i] + b[j][i];
                if (act == kActSilu) {
                    const float s = sigmoid(o);
                    d[j][i] *= s * (1.f + o * (1.f - s));
                }
                if (act == kActGatePost) {
                    const float s = sigmoid(zv[j][i]);
                    gz[i] = d[j][i] * o * s * (1.f + zv[j][i] * (1.f - s));
                    d[j][i] *= zv[j][i] * s;
                }
                dw[j][i] += d[j][i] * u[j][i];
                db[j][i] += d[j][i];
                d[j][i] *= w[j][i];
                sn += d[j][i];
                snh += d[j][i] * u[j][i];
            }
            if (act == kActGatePost && in[j]) store_vec<V>(dz + base + (j * tpg + lane) * V, gz);
        }
        snh = group_sum(snh, tpg, part) / (float)n;
        sn = center ? group_sum(sn, tpg, part) / (float)n : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (!in[j]) continue;
            float gx[V], gz[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                gx[i] = r * (d[j][i] - sn - u[j][i] * snh);
                if (act == kActGatePre) {
                    const float s = sigmoid(zv[j][i]);
                    gz[i] = gx[i] * xv[j][i] * s * (1.f + zv[j][i] * (1.f - s));
                    gx[i] *= zv[j][i] * s;
                }
            }
            store_vec<V>(dx + base + (j * tpg + lane) * V, gx);
            if (act == kActGatePre) store_vec<V>(dz + base + (j * tpg + lane) * V, gz);
        }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int e = (j * tpg + lane) * V;
        if (mine && e < n) {
            if (dwp) store_vec<V>(dwp + (size_t)row * C + c0 + e, dw[j]);
            if (dbp) store_vec<V>(dbp + (size_t)row * C + c0 + e, db[j]);
        }
    }
}

// Sums of the partial rows of dw (blockIdx.y 0) and db (1): 64 channels a workgroup, 16 runs
// of rows, then the runs in their order.
__global__ __launch_bounds__(1024) void norm_params_kernel(const float* __restrict__ dwp,
                                                           const float* __restrict__ dbp, float* __restrict__ dw,
                                                           float* __restrict__ db, int C, int rows) {
    __shared__ float run[16][64];
    const float* src = blockIdx.y ? dbp : dwp;
    float* dst = blockIdx.y ? db : dw;
    if (!dst) return;
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6;
    float s = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int r = k; r < rows; r += 16) s += src[(size_t)r * C + c];
    }
    run[k][threadIdx.x & 63] = s;
    __syncthreads();
    if (k == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += run[i][threadIdx.x];
        dst[c] = s;
    }
}

namespace {

// Threads a group (a power of two), vectors a thread and channels a vector (n at most 16384). `wide`:
// vectors of eight, 16 bytes of bf16; fp32 goes by four, so that neighbours' accesses touch. Among the
// counts of vectors a thread may hold, the one that leaves the fewest threads without a channel; where few
// groups are to be normed, the one that gives each the most threads.
struct NormPlan {
    int vec, k, tpg, threads;
};
NormPlan norm_plan(int n, long slots, bool wide) {
    NormPlan p;
    p.vec = n % 8 == 0 && wide ? 8 : n % 4 == 0 ? 4 : 1;
    const int m = n / p.vec;
    double best = 0;
    for (int k : {1, 2, 3, 5, 16}) {
        if (k == 16 && p.vec != 1) continue;
        int tpg = 1;
        while (tpg * k < m) tpg *= 2;
        if (tpg > 1024 || (tpg > 256 && k == 16 && best > 0)) continue;
        const double use = slots * tpg < 65536 ? 1.0 / k : (double)m / (tpg * k) - (k == 16 ? 0.2 : 0);
        if (use > best + 1e-9) {
            best = use;
            p.k = k;
            p.tpg = tpg;
        }
    }
    p.threads = p.tpg > 256 ? p.tpg : 256;
    return p;
}

struct NormRows {
    int gpw, tpw, gblocks, tblocks;
};
NormRows norm_rows(const NormPlan& p, long tokens, int groups) {
    const int ns = p.threads / p.tpg;
    NormRows r = {1, 1, 1, 1};
    double best = 0;
    for (int gpw = 1; gpw <= std::min(ns, groups); ++gpw) {
        const int tpw = ns / gpw, blocks = (groups + gpw - 1) / gpw;
        const double use = (double)groups / ((double)blocks * gpw) * (gpw * tpw) / ns;
        if (use >= best - 1e-9) {
            best = use;
            r.gpw = gpw;
            r.tpw = tpw;
            r.gblocks = blocks;
        }
    }
    const long turns = (tokens + r.tpw - 1) / r.tpw;
    // As many workgroups as the compute units hold at once, which the registers for a thread's channels decide: four
    // with up to five channels a thread, three with twelve, two with more or with 1024 threads (eight channels: two
    // and four take the same time). In us with 512, 768 and 1024 workgroups: 16000 x 1024 in one group (four channels)
    // 88, 66, 59; 8000 x 1683 in 9 (three) 101, 71, 59; 16000 x 2700 in one (twelve) 195, 154, 201; 16000 x 2048 in one
    // (eight) 118, 145, 118; 16384 x 5120 in 8 (twenty) 284, 361, 294.
    const int held = p.vec * p.k;
    const long want = std::max(1L, (p.threads > 256 ? 512L : held <= 5 ? 1024L : held == 12 ? 768L : 512L) / r.gblocks);
    r.tblocks = (int)std::max(1L, std::min(std::min(turns, want), std::max(1L, 2048L / r.tpw)));
    return r;
}

// The instances norm_plan() reaches.
template <int V, int NTHR, typename F> hipError_t by_k(const NormPlan& p, F&& f) {
    using std::integral_constant;
    const integral_constant<int, V> v;
    const integral_constant<int, NTHR> t;
    switch (p.k) {
        case 1: return f(v, integral_constant<int, 1>{}, t);
        case 2: return f(v, integral_constant<int, 2>{}, t);
        case 3: return f(v, integral_constant<int, 3>{}, t);
        case 5: return f(v, integral_constant<int, 5>{}, t);
    }
    if constexpr (V == 1)
        if (p.k == 16) return f(v, integral_constant<int, 16>{}, t);
    return hipErrorInvalidValue;
}
template <bool WIDE, typename F> hipError_t by_plan(const NormPlan& p, F&& f) {
    if constexpr (WIDE)
        if (p.vec == 8) return p.threads <= 256 ? by_k<8, 256>(p, f) : by_k<8, 1024>(p, f);
    if (p.vec == 4) return p.threads <= 256 ? by_k<4, 256>(p, f) : by_k<4, 1024>(p, f);
    return p.threads <= 256 ? by_k<1, 256>(p, f) : by_k<1, 1024>(p, f);
}
template <typename F> hipError_t by_type(int dt, F&& f) { return dt == kBF16 ? f(bf16()) : f(float()); }

}  // namespace

hipError_t launch_group_norm(const NormArgs& a, hipStream_t stream) {
    const int n = a.channels / a.groups;
    const long slots = a.tokens * a.groups;
    const NormPlan p = norm_plan(n, slots, a.x_dtype == kBF16);
    const long per = p.threads / p.tpg;
    return by_type(a.x_dtype, [&](auto tx) {
        return by_type(a.z_dtype, [&](auto tz) {
            return by_type(a.out_dtype, [&](auto to) {
                using TX = decltype(tx);
                using TZ = decltype(tz);
                using TO = decltype(to);
                return by_plan<sizeof(TX) == 2>(p, [&](auto v, auto k, auto nt) {
                    group_norm_kernel<TX, TZ, TO, decltype(v)::value, decltype(k)::value, decltype(nt)::value>
                        <<<dim3((unsigned)((slots + per - 1) / per)), p.threads, 0, stream>>>(
                            (const TX*)a.x, (const TZ*)a.z, a.weight, a.bias, (TO*)a.out, slots, a.groups, n,
                            p.tpg, a.act, a.center, a.eps);
                    return hipGetLastError();
                });
            });
        });
    });
}

int group_norm_rows(long tokens, int channels, int groups) {
    const NormRows r = norm_rows(norm_plan(channels / groups, tokens * groups, false), tokens, groups);
    return r.tblocks * r.tpw;
}

hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream) {
    const int n = a.channels / a.groups;
    const NormPlan p = norm_plan(n, a.tokens * a.groups, false);
    const NormRows r = norm_rows(p, a.tokens, a.groups);
    hipError_t e = by_type(a.x_dtype, [&](auto tx) {
        return by_type(a.z_dtype, [&](auto tz) {
            return by_plan<false>(p, [&](auto v, auto k, auto nt) {
                using TX = decltype(tx);
                using TZ = decltype(tz);
                group_norm_backward_kernel<TX, TZ, decltype(v)::value, decltype(k)::value, decltype(nt)::value>
                    <<<dim3(r.gblocks, r.tblocks), p.threads, 0, stream>>>(
                        (const TX*)a.x, (const TZ*)a.z, a.weight, a.bias, a.dy, a.dx, a.dz,
                        a.dweight ? a.dwp : nullptr, a.dbias ? a.dbp : nullptr, a.tokens, a.groups, n, p.tpg,
                        a.act, a.center, a.eps, r.gpw, r.tpw, r.tblocks);
                return hipGetLastError();
            });
        });
    });
    if (e != hipSuccess || !(a.dweight || a.dbias)) return e;
    norm_params_kernel<<<dim3((a.channels + 63) / 64, 2), 1024, 0, stream>>>(a.dwp, a.dbp, a.dweight, a.dbias,
                                                                           a.channels, r.tblocks * r.tpw);
    return hipGetLastError();
}

hipError_t launch_norm_params_zero(const NormArgs& a, hipStream_t stream) {
    if (!(a.dweight || a.dbias)) return hipSuccess;
    norm_params_kernel<<<dim3((a.channels + 63) / 64, 2), 1024, 0, stream>>>(nullptr, nullptr, a.dweight, a.dbias,
                                                                           a.channels, 0);
    return hipGetLastError();
}

}  // namespace ssd

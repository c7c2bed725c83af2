// The norm before a layer, with the residual addition in front of it, and its gradient.
//
// Forward, for each row t:  s = x + r (stored in the row's type; s = x without a residual),
//   mu = mean(s) (0 in the root-mean-square form), q = 1 / sqrt(mean((s - mu)^2) + eps),
//   y = (s - mu) q w + b.
// Backward, with xh = (s - mu) q and u = dy w:
//   dx = q (u - mean(u) - xh mean(u xh)) + dr   (no mean(u) in the root-mean-square form),
//   dw = sum_t dy xh,  db = sum_t dy.
#include "f32x2.cuh"
#include "moe_internal.cuh"

namespace rdg {
namespace {

constexpr int kMaxRowBytes = 32768;  // 1024 threads x 2 vectors of 16 bytes
constexpr int kWarpRowBytes = 1024;  // rows up to this take one warp each
constexpr int kWarps = 8;            // warps of a block in that form
constexpr int V = 2;                 // 16-byte vectors of a row in a thread's hands
constexpr int kStages = 2;           // rows a thread group has in flight or in hand
constexpr int kFlight = 30 << 10;    // bytes of rows on their way to an SM in the forward pass
constexpr float kInfinity = __builtin_huge_valf();
constexpr float kLeastVar = 1e-30f;  // squares that count lose digits below it (fp32's range ends)

template <typename T>
struct Vec;  // 16 bytes of a row as pairs of fp32 values
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8, P = 4;
    static __device__ __forceinline__ void unpack(uint4 u, f2* f) {
        f[0] = unpack_bf16x2(u.x);
        f[1] = unpack_bf16x2(u.y);
        f[2] = unpack_bf16x2(u.z);
        f[3] = unpack_bf16x2(u.w);
    }
    static __device__ __forceinline__ uint32_t pack2(f2 f) {
        float lo, hi;
        split(f, lo, hi);
        return pack_bf16x2(lo, hi);
    }
    static __device__ __forceinline__ uint4 pack(const f2* f) {
        return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4, P = 2;
    static __device__ __forceinline__ void unpack(uint4 u, f2* f) {
        f[0] = make_f2(__uint_as_float(u.x), __uint_as_float(u.y));
        f[1] = make_f2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 pack(const f2* f) {
        float4 v;
        split(f[0], v.x, v.y);
        split(f[1], v.z, v.w);
        return make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                          __float_as_uint(v.w));
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Keeps the compiler from holding values unpacked from u over this point.
__device__ __forceinline__ void keep_packed(uint4& u) {
    asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
}

// N weights (fp32 or bf16) from column c on; `fill` where there are none
template <int N>
__device__ __forceinline__ void load_params(const void* p, bool bf16, int c, float fill, f2* f) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if (p == nullptr) {
            f[i / 2] = f[i / 2 + 1] = both(fill);
        } else if (bf16) {
            const uint2 u = *reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(p) + c + i);
            f[i / 2] = unpack_bf16x2(u.x);
            f[i / 2 + 1] = unpack_bf16x2(u.y);
        } else {
            Vec<float>::unpack(
                *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + c + i), f + i / 2);
        }
    }
}
__device__ __forceinline__ float halves_sum(f2 a) {
    float lo, hi;
    split(a, lo, hi);
    return lo + hi;
}

// sum / n: the product with 1 / n, and its remainder put right, so that a row of equal values has
// that value as its mean (sum / n exactly; the product alone misses it for 1000 values, say, and
// rstd makes the difference large).
__device__ __forceinline__ float mean_of(float sum, float n, float inv) {
    const float m = sum * inv;
    return fmaf(fmaf(-m, n, sum), inv, m);
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(at)
                 : "memory");
    return u;
}
__device__ __forceinline__ void sts128(uint32_t at, uint4 u) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(u.x), "r"(u.y), "r"(u.z),
                 "r"(u.w)
                 : "memory");
}

// Sums of K values over the threads that share a row: the lanes of a warp, or the whole block
// through shared memory. `red` holds two buffers of K x 32 floats used in turn, so that one
// barrier a sum is enough: a buffer is written again only after the next sum's barrier. After it
// every thread adds the warps' sums itself (broadcast loads: shorter than another tree of
// shuffles); places without a warp stay 0.
template <int THREADS, bool WARP, int K>
struct RowSum {
    static constexpr int kFloats = WARP ? 4 : 2 * K * 32;
    float* red;
    int turn = 0;
    __device__ __forceinline__ explicit RowSum(float* r) : red(r) {
        if constexpr (!WARP) {
            for (int i = threadIdx.x; i < kFloats; i += blockDim.x) red[i] = 0.f;
            __syncthreads();
        }
    }
    __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if constexpr (!WARP) {
            float* buf = red + turn;
            turn ^= K * 32;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int k = 0; k < K; ++k) buf[k * 32 + (threadIdx.x >> 5)] = v[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                f2 t = both(0.f);
#pragma unroll
                for (int w = 0; w < THREADS / 32; w += 4) {
                    f2 q[2];
                    Vec<float>::unpack(*reinterpret_cast<const uint4*>(buf + k * 32 + w), q);
                    t = add(t, add(q[0], q[1]));
                }
                v[k] = halves_sum(t);
            }
        }
    }
};

struct NormArgs {
    const void* x;
    const void* residual;  // or NULL
    const void* weight;    // or NULL: 1
    const void* bias;      // or NULL: 0
    void* sum;             // with a residual
    void* y;
    float* mean;           // or NULL
    float* rstd;           // or NULL
    int T, d;
    float eps;
    bool param_bf16;
};

// A thread's share of the rows, in both kernels. Rows go to thread groups (a warp, or the block)
// in turn; a thread holds V vectors of its row, its weights stay in registers, and its vectors of
// the next row are on their way to its own places in shared memory meanwhile (cp.async: no
// barrier, each thread reads what it copied). Two stages: with three or more the norm of 16384
// rows of 10 KB took 58 to 61 us instead of 52. Vectors past the row's end are zeros that were
// stored once, so that the loop over them has no branch.
template <int A, bool WARP>
struct Share {
    int gt, nv;
    bool ok[V];
    uint32_t plane, place;         // bytes from one vector's places to the next's; the first's
    long long row, stride, at, step;  // at: this thread's first vector of the row
    int T;
    __device__ __forceinline__ Share(int T_, int nv_, uint4* ring) : nv(nv_), T(T_) {
        gt = WARP ? (threadIdx.x & 31) : threadIdx.x;
        const int width = WARP ? 32 : blockDim.x, groups = WARP ? kWarps : 1;
        row = (long long)blockIdx.x * groups + (WARP ? threadIdx.x >> 5 : 0);
        stride = (long long)gridDim.x * groups;
        at = row * nv + gt;
        step = stride * nv;
        plane = blockDim.x * 16;
        place = smem_u32(ring) + threadIdx.x * 16;
        apart = width;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            ok[i] = gt + i * width < nv;
            if (!ok[i])
#pragma unroll
                for (int k = 0; k < 2 * A; ++k)
                    sts128(place + (k * V + i) * plane, make_uint4(0, 0, 0, 0));
        }
    }
    int apart;                     // vectors between a thread's first and second
    __device__ __forceinline__ int column(int i) const { return gt + i * apart; }
    __device__ __forceinline__ uint4 load(uint32_t stage, int which, int i) const {
        return lds128(stage + (which * V + i) * plane);
    }
    // The row `rows` steps on, into the places from `stage` on.
    __device__ __forceinline__ void fetch(const uint4* const (&src)[A], int rows, uint32_t stage) {
        if (row + rows * stride < T) {
            const long long from = at + rows * step;
#pragma unroll
            for (int k = 0; k < A; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (ok[i]) cp_async16(stage + (k * V + i) * plane, src[k] + from + i * apart);
        }
        cp_async_commit();
    }
    __device__ __forceinline__ void next() {
        row += stride;
        at += step;
    }
};

// Bound by memory: 2 or 4 values of the row's type read and written for each of T d, and the
// statistics. 16384 rows of 5120 bf16 values, root mean square: 52 us, 6.4 TB/s (0.95 of the
// measured copy bandwidth); 4096 rows of 4096, layer norm with residual: 24.2 us, 5.6 TB/s, where
// starting and draining count for more; 8192 rows of 2880 fp32 values, layer: 34.6 us (0.81);
// 16384 of 512 bf16 values, a warp a row, rms: 6.0 us (0.83); 8 rows of 2048: 1.8 us, latency
// alone. The layer norm's
// two sums over a row are taken one after the other (the squares about the mean, so that a large
// mean costs no precision); the second costs 2 us of those 24.2.
// The bound on blocks holds the registers at 64 (80 where a warp takes a row): the rare second
// pass over a row out of range would have 82 otherwise. It costs other rows 0 to 2%.
template <typename T, int THREADS, bool RMS, bool RES>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : THREADS == 256 ? 3 : 1)
    norm_kernel(const NormArgs a) {
    constexpr int N = Vec<T>::N, P = Vec<T>::P, A = RES ? 2 : 1;
    constexpr bool WARP = THREADS == 32 * kWarps;
    using Sum = RowSum<THREADS, WARP, 1>;
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[Sum::kFloats];
    Share<A, WARP> t(a.T, a.d / N, ring);
    const uint4* src[A];
    src[0] = static_cast<const uint4*>(a.x);
    if (RES) src[A - 1] = static_cast<const uint4*>(a.residual);
    uint4* y = static_cast<uint4*>(a.y);
    uint4* sum = static_cast<uint4*>(a.sum);
    uint32_t stage = t.place, other = t.place + A * V * t.plane;

    griddep_wait();
    t.fetch(src, 0, stage);
    f2 w[V * P], b[V * P];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (t.ok[i]) {
            load_params<N>(a.weight, a.param_bf16, t.column(i) * N, 1.f, w + i * P);
            if (!RMS) load_params<N>(a.bias, a.param_bf16, t.column(i) * N, 0.f, b + i * P);
        }
    Sum total(red);
    const float inv = 1.f / (float)a.d;
    for (; t.row < a.T; t.next()) {
        t.fetch(src, 1, other);
        cp_async_wait<1>();
        f2 f[V * P];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Vec<T>::unpack(t.load(stage, 0, i), f + i * P);
            if constexpr (RES) {
                f2 r[P];
                Vec<T>::unpack(t.load(stage, 1, i), r);
#pragma unroll
                for (int j = 0; j < P; ++j) f[i * P + j] = add(f[i * P + j], r[j]);
                const uint4 u = Vec<T>::pack(f + i * P);
                if (t.ok[i]) sum[t.at + i * t.apart] = u;
                Vec<T>::unpack(u, f + i * P);  // the norm sees the stored sum
            }
        }
        // f less its mean mu; returns the sum of its squares.
        float mu = 0.f;
        auto centre = [&] {
            float v[1];
            f2 s = both(0.f);
            if constexpr (!RMS) {
#pragma unroll
                for (int j = 0; j < V * P; ++j) s = add(s, f[j]);
                v[0] = halves_sum(s);
                total(v);
                mu = mean_of(v[0], (float)a.d, inv);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const f2 minus = both(t.ok[i] ? -mu : 0.f);
#pragma unroll
                    for (int j = 0; j < P; ++j) f[i * P + j] = add(f[i * P + j], minus);
                }
                s = both(0.f);
            }
#pragma unroll
            for (int j = 0; j < V * P; ++j) s = fma(f[j], f[j], s);
            v[0] = halves_sum(s);
            total(v);
            return v[0];
        };
        float var = fmaf(centre(), inv, a.eps), q = 1.f / sqrtf(var), rstd = q;
        // Squares (or the sum) beyond fp32, or below it with an eps of next to nothing: once more
        // with the row scaled by a power of two. What is not finite then holds NaN or an infinity.
        // All threads of a row have the same var.
        if (__builtin_expect(!(var >= kLeastVar && var < kInfinity), 0)) {
            const bool small = var < kLeastVar;
            const float up = small ? 0x1p96f : 0x1p-100f, down = small ? 0x1p-96f : 0x1p100f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                Vec<T>::unpack(t.load(stage, 0, i), f + i * P);
                if constexpr (RES) {
                    f2 r[P];
                    Vec<T>::unpack(t.load(stage, 1, i), r);
#pragma unroll
                    for (int j = 0; j < P; ++j) f[i * P + j] = add(f[i * P + j], r[j]);
                    Vec<T>::unpack(Vec<T>::pack(f + i * P), f + i * P);
                }
#pragma unroll
                for (int j = 0; j < P; ++j) f[i * P + j] = mul(f[i * P + j], both(up));
            }
            var = fmaf(centre(), inv, a.eps * up * up);
            q = var < kInfinity ? 1.f / sqrtf(var) : __int_as_float(0x7fffffff);
            rstd = q * up;
            mu *= down;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f2 o[P];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                o[j] = mul(f[i * P + j], both(q));
                o[j] = RMS ? mul(o[j], w[i * P + j]) : fma(o[j], w[i * P + j], b[i * P + j]);
            }
            if (t.ok[i]) y[t.at + i * t.apart] = Vec<T>::pack(o);
        }
        if (t.gt == 0) {
            if (!RMS && a.mean) a.mean[t.row] = mu;
            if (a.rstd) a.rstd[t.row] = rstd;
        }
        const uint32_t was = stage;
        stage = other;
        other = was;
    }
}

// Resident blocks that the backward kernel's registers are bounded for: fp32 rows have half as many
// sums in a thread. (1021 rows of 2880 fp32 values: 14.1 us with one block of 384, 11.8 with two.)
constexpr int min_blocks(int threads, size_t element) {
    return threads <= 320 ? (element == 4 ? 3 : 2) : threads <= 512 && element == 4 ? 2 : 1;
}

struct NormBackwardArgs {
    const void* dy;
    const void* x;
    const void* weight;     // or NULL: 1
    const float* mean;      // NULL in the root-mean-square form
    const float* rstd;
    const void* dresidual;  // or NULL
    void* dx;
    float* part;            // [blocks, 2, d]: this block's dw and db, or NULL
    int* status;
    int T, d;
    bool param_bf16;
};

// As the forward kernel; a thread keeps the sums of its columns' dw and db in registers over all
// its rows. The row's vectors stay packed until the two sums over the row are known and are
// unpacked again: holding them as fp32 would cost 32 registers, and so a resident block.
// Bound by memory (3 or 4 values for each of T d), closely followed by issue: half of all slots at
// 16384 rows of 5120 bf16 values with a residual's gradient, 106 us with the reduction, 6.3 TB/s
// (0.93 of the measured copy bandwidth). With scalar arithmetic and branches on the row's end it
// took 200 us. Narrow rows pay more for the partial sums (4096 rows of 2048: 19 us, floor 10).
template <typename T, int THREADS, bool RMS, bool RES>
__global__ void __launch_bounds__(THREADS, min_blocks(THREADS, sizeof(T)))
    norm_backward_kernel(const NormBackwardArgs a) {
    constexpr int N = Vec<T>::N, P = Vec<T>::P, A = RES ? 3 : 2;
    constexpr bool WARP = THREADS == 32 * kWarps;
    using Sum = RowSum<THREADS, WARP, 2>;
    // Whether mean(u) goes into u, an instruction less, or, times q, into what is added last. The
    // first is faster for bf16 rows of up to 10 KB with a residual's gradient (16384 rows of 5120:
    // 106 us, 120 the other way), the second for the others, by registers (8192 rows of 2880 fp32
    // values: 49 us, 58 the other way; 4096 of 16384 bf16 values with a residual's: 144 and 177).
    constexpr bool kMeanInU = RES && sizeof(T) == 2 && THREADS <= 320;
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[Sum::kFloats];
    Share<A, WARP> t(a.T, a.d / N, ring);
    const uint4* src[A];
    src[0] = static_cast<const uint4*>(a.dy);
    src[1] = static_cast<const uint4*>(a.x);
    if (RES) src[A - 1] = static_cast<const uint4*>(a.dresidual);
    uint4* dx = static_cast<uint4*>(a.dx);
    uint32_t stage = t.place, other = t.place + A * V * t.plane;

    griddep_wait();
    griddep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = MOE_OK;  // nothing here can go wrong
    t.fetch(src, 0, stage);
    f2 w[V * P], dw[V * P], db[V * P];
#pragma unroll
    for (int j = 0; j < V * P; ++j) w[j] = dw[j] = db[j] = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (t.ok[i]) load_params<N>(a.weight, a.param_bf16, t.column(i) * N, 1.f, w + i * P);
    Sum total(red);
    const float inv = 1.f / (float)a.d;
    float mu = 0.f, q = 0.f;
    if (t.row < a.T) {
        if (!RMS) mu = a.mean[t.row];
        q = a.rstd[t.row];
    }
    for (; t.row < a.T; t.next()) {
        t.fetch(src, 1, other);
        float mu2 = 0.f, q2 = 0.f;  // the next row's
        if (t.row + t.stride < a.T) {
            if (!RMS) mu2 = a.mean[t.row + t.stride];
            q2 = a.rstd[t.row + t.stride];
        }
        cp_async_wait<1>();
        uint4 pd[V], px[V];
        f2 t0 = both(0.f), t1 = t0;
        // The mean is subtracted before q multiplies: x q - mu q, with mu q rounded, would shift the
        // whole row by up to 2^-25 |mu| q.
        const f2 fq = both(q), minus_mu = both(-mu);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            pd[i] = t.load(stage, 0, i);
            px[i] = t.load(stage, 1, i);
            f2 g[P], x[P];
            Vec<T>::unpack(pd[i], g);
            Vec<T>::unpack(px[i], x);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int k = i * P + j;
                const f2 xh = mul(RMS ? x[j] : add(x[j], minus_mu), fq), u = mul(g[j], w[k]);
                dw[k] = fma(g[j], xh, dw[k]);
                t0 = fma(u, xh, t0);
                if (!RMS) {
                    db[k] = add(db[k], g[j]);
                    t1 = add(t1, u);
                }
            }
        }
        float v[2] = {halves_sum(t0), RMS ? 0.f : halves_sum(t1)};
        total(v);
        const f2 minus_m1 = both(-v[1] * inv), minus_m2 = both(-v[0] * inv);
        const f2 minus_m1q = both(-v[1] * inv * q);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            keep_packed(pd[i]);
            keep_packed(px[i]);
            f2 g[P], x[P], o[P];
            Vec<T>::unpack(pd[i], g);
            Vec<T>::unpack(px[i], x);
            if constexpr (RES) Vec<T>::unpack(t.load(stage, 2, i), o);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const f2 xh = mul(RMS ? x[j] : add(x[j], minus_mu), fq);
                if (RMS || kMeanInU) {
                    const f2 u = RMS ? mul(g[j], w[i * P + j]) : fma(g[j], w[i * P + j], minus_m1);
                    const f2 e = fma(xh, minus_m2, u);
                    o[j] = RES ? fma(e, fq, o[j]) : mul(e, fq);
                } else {
                    const f2 e = fma(xh, minus_m2, mul(g[j], w[i * P + j]));
                    o[j] = fma(e, fq, RES ? add(o[j], minus_m1q) : minus_m1q);
                }
            }
            if (t.ok[i]) dx[t.at + i * t.apart] = Vec<T>::pack(o);
        }
        const uint32_t was = stage;
        stage = other;
        other = was;
        mu = mu2;
        q = q2;
    }
    if (a.part == nullptr) return;
    constexpr int K = RMS ? 1 : 2;  // dw, and db
    float* part = a.part + (size_t)blockIdx.x * K * a.d;
    float* to = part;
    if constexpr (WARP) {  // the block's warps first, in order
        cp_async_wait<0>();
        __syncthreads();
        to = reinterpret_cast<float*>(ring) + (threadIdx.x >> 5) * K * a.d;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (t.ok[i])
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                const int c = t.column(i) * N + j, k = (i * N + j) / 2;
                *reinterpret_cast<uint4*>(to + c) = Vec<float>::pack(dw + k);
                if (!RMS) *reinterpret_cast<uint4*>(to + a.d + c) = Vec<float>::pack(db + k);
            }
    if constexpr (WARP) {
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(ring);
        for (int c = threadIdx.x; c < K * a.d; c += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += all[k * K * a.d + c];
            part[c] = s;
        }
    }
}

// dw (and db): the blocks' partial sums [P, columns] added in a fixed order, columns = d or 2 d.
// They lie in L2 (12 MB at d = 5120); the kernel starts while the blocks before it finish and is
// latency for the most part (1021 rows of 2880 fp32 values: 11.8 us in all with 16 warps a block,
// 11.0 with 32).
// A block takes 64 columns; its 32 warps take rows 32 apart, eight loads in flight each.
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(32 * kReduceWarps)
    norm_reduce_kernel(const float* __restrict__ part, int P, int d, int columns,
                       float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float2 s[kReduceWarps][32];
    const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * 2;  // d is a multiple of 4: no pair spans dw and db
    float2 t = make_float2(0.f, 0.f);
    griddep_wait();
    if (c < columns) {
#pragma unroll 8
        for (int p = wy; p < P; p += kReduceWarps) {
            const float2 v = *reinterpret_cast<const float2*>(part + (size_t)p * columns + c);
            t.x += v.x;
            t.y += v.y;
        }
    }
    s[wy][lane] = t;
    __syncthreads();
    if (wy == 0 && c < columns) {
#pragma unroll
        for (int k = 1; k < kReduceWarps; ++k) {
            t.x += s[k][lane].x;
            t.y += s[k][lane].y;
        }
        float* out = c < d ? dweight : dbias;
        if (out) *reinterpret_cast<float2*>(out + (c < d ? c : c - d)) = t;
    }
}

// How the rows of d values are taken: by a warp each (threads = 32 kWarps), or by a block each.
struct Shape {
    bool warp;
    int threads;
};
Shape shape_of(int d, bool bf16) {
    const int bytes = d * (bf16 ? 2 : 4), nv = bytes / 16;
    Shape s;
    s.warp = bytes <= kWarpRowBytes;
    s.threads = s.warp ? 32 * kWarps : ((nv + V - 1) / V + 31) / 32 * 32;
    return s;
}

// Calls f.run with the row type, the thread bound, RMS and RES as compile-time values.
template <typename T, int THREADS, typename F>
cudaError_t with_flags(bool rms, bool res, const F& f) {
    if (rms)
        return res ? f.template run<T, THREADS, true, true>()
                   : f.template run<T, THREADS, true, false>();
    return res ? f.template run<T, THREADS, false, true>()
               : f.template run<T, THREADS, false, false>();
}
template <typename T, typename F>
cudaError_t with_threads(const Shape& s, bool rms, bool res, const F& f) {
    if (s.warp) return with_flags<T, 32 * kWarps>(rms, res, f);
    if constexpr (F::kTwoBlocks)
        if (s.threads <= 320) return with_flags<T, 320>(rms, res, f);
    return s.threads <= 512 ? with_flags<T, 512>(rms, res, f) : with_flags<T, 1024>(rms, res, f);
}
template <typename F>
cudaError_t with_types(bool bf16, const Shape& s, bool rms, bool res, const F& f) {
    return bf16 ? with_threads<__nv_bfloat16>(s, rms, res, f)
                : with_threads<float>(s, rms, res, f);
}

constexpr int kMaxSmem = 6 * kMaxRowBytes;

int groups_of(int T, const Shape& s) { return s.warp ? (T + kWarps - 1) / kWarps : T; }

struct Forward {
    static constexpr bool kTwoBlocks = false;
    const NormArgs& a;
    Shape s;
    cudaStream_t stream;
    template <typename T, int THREADS, bool RMS, bool RES>
    cudaError_t run() const {
        auto fn = norm_kernel<T, THREADS, RMS, RES>;
        const int smem = kStages * (RES ? 2 : 1) * V * s.threads * 16;
        cudaError_t e = ensure_max_dynamic_smem((const void*)fn, kMaxSmem);
        if (e != cudaSuccess) return e;
        // Blocks an SM: as many as have about 30 KB of rows on their way. More of them get less from
        // memory: 16384 rows of 4096 with a residual took 95 us with four blocks, 85 with two; of
        // 5120 without one 57 with two and 52 with three. With few rows a block the last round
        // counts more: 4096 rows took 24.3 us with four blocks, 25.0 with two.
        const int flight = smem / kStages;
        int of_sm = (kFlight + flight - 1) / flight;
        if (a.T < 24 * of_sm * device_sm_count()) of_sm *= 2;
        int most = resident_blocks((const void*)fn, s.threads, smem);
        if (!s.warp && most > of_sm * device_sm_count()) most = of_sm * device_sm_count();
        const int need = groups_of(a.T, s);
        return launch_kernel(fn, dim3(need < most ? need : most), dim3(s.threads), smem, stream, a);
    }
};

// Blocks of the backward pass at most, and so partial sums of dw and db: 640 threads an SM, two
// blocks at least (16384 rows of 1024 bf16 values: 39 us with four blocks of 64 threads, 32 with
// ten).
int backward_max_blocks(int T, const Shape& s) {
    const int of_sm = 640 / s.threads > 2 ? 640 / s.threads : 2;
    const int need = groups_of(T, s), most = device_sm_count() * of_sm;
    return need < most ? need : most;
}

struct Backward {
    static constexpr bool kTwoBlocks = true;  // blocks of at most 320 threads: two an SM
    const NormBackwardArgs& a;
    Shape s;
    float* dweight;
    float* dbias;
    cudaStream_t stream;
    template <typename T, int THREADS, bool RMS, bool RES>
    cudaError_t run() const {
        auto fn = norm_backward_kernel<T, THREADS, RMS, RES>;
        int smem = kStages * (RES ? 3 : 2) * V * s.threads * 16;
        if (s.warp && smem < kWarps * 2 * a.d * 4) smem = kWarps * 2 * a.d * 4;
        cudaError_t e = ensure_max_dynamic_smem((const void*)fn, kMaxSmem);
        if (e != cudaSuccess) return e;
        int blocks = resident_blocks((const void*)fn, s.threads, smem);
        const int most = backward_max_blocks(a.T, s);
        if (blocks > most) blocks = most;
        e = launch_kernel(fn, dim3(blocks), dim3(s.threads), smem, stream, a);
        if (e != cudaSuccess || a.part == nullptr) return e;
        PdlScope pdl(true);
        const int columns = RMS ? a.d : 2 * a.d;
        return launch_kernel(norm_reduce_kernel, dim3((columns + 63) / 64),
                             dim3(32 * kReduceWarps), 0, stream, (const float*)a.part, blocks, a.d,
                             columns, dweight, dbias);
    }
};

}  // namespace

bool norm_row_fits(int d, bool bf16) { return (size_t)d * (bf16 ? 2 : 4) <= kMaxRowBytes; }

size_t norm_backward_scratch_bytes(int T, int d, bool bf16) {
    return (size_t)backward_max_blocks(T, shape_of(d, bf16)) * 2 * d * 4;
}

cudaError_t launch_norm(const void* x, const void* residual, bool bf16, int T, int d,
                        const void* weight, const void* bias, bool param_bf16, float eps, bool rms,
                        void* sum, void* y, float* mean, float* rstd, cudaStream_t s) {
    const NormArgs a = {x, residual, weight, bias, sum, y, mean, rstd, T, d, eps, param_bf16};
    const Shape sh = shape_of(d, bf16);
    return with_types(bf16, sh, rms, residual != nullptr, Forward{a, sh, s});
}

cudaError_t launch_norm_backward(const void* dy, const void* x, bool bf16, int T, int d,
                                 const void* weight, bool param_bf16, const float* mean,
                                 const float* rstd, const void* dresidual, bool rms, void* dx,
                                 float* dweight, float* dbias, float* part, int* status,
                                 cudaStream_t s) {
    const NormBackwardArgs a = {dy, x, weight, mean, rstd, dresidual, dx,
                                dweight || dbias ? part : nullptr, status, T, d, param_bf16};
    const Shape sh = shape_of(d, bf16);
    return with_types(bf16, sh, rms, dresidual != nullptr,
                      Backward{a, sh, dweight, dbias, s});
}

}  // namespace rdg

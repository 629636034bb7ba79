// moe_train.cu -- the row-wise operators of a training step around the
// expert FFN: the gradients of the combine ("local sum"), of the permute and
// of the top-K gate, and the norms before and after the block (with the
// block's gate and residual scale, fused with the combine) with their
// gradient.  All are bound by device memory at training sizes and by latency
// at decode sizes: each reads its rows once, keeps its sums in fp32 and rounds
// each output once.  Times in this file are of calls back to back, inputs larger
// than L2, unless said otherwise.
#include <atomic>
#include <climits>
#include <type_traits>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {

namespace {

int launched(cudaError_t e) {
    count_launch();
    if (e != cudaSuccess) {
        cudaGetLastError();
        return -3;
    }
    return 0;
}

template <typename T>
__device__ __forceinline__ void up(const int4& v, float* f) {
    unpack(v, f, (const T*)nullptr);
}
template <typename T>
__device__ __forceinline__ int4 down(const float* f) {
    return pack(f, (const T*)nullptr);
}

// ------------------------------------------------------------ block sums
// Eight sums over a warp in nine shuffles: each step halves the values a lane
// holds and doubles the lanes behind each; lane l ends with the sum of value
// l & 7.
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane) {
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool hi = lane & 4;
        const float send = hi ? v[i] : v[i + 4];
        a[i] = (hi ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, send, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool hi = lane & 2;
        const float send = hi ? a[i] : a[i + 2];
        b[i] = (hi ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, send, 2);
    }
    {
        const bool hi = lane & 1;
        const float send = hi ? b[0] : b[1];
        c = (hi ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, send, 1);
    }
    c += __shfl_xor_sync(0xffffffffu, c, 8);
    c += __shfl_xor_sync(0xffffffffu, c, 16);
    return c;
}

// Eight sums over the block, given to every thread.  `buf` is [32][8] floats,
// zero past the block's warps, so that sixteen warps' are read at once; two
// calls may not share it without a barrier in between (callers alternate two
// buffers, so one barrier per call is enough).
__device__ __forceinline__ void block_sum8(float (&v)[8], float* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float c = warp_sum8(v, lane);
    if (nw > 1) {
        if (lane < 8) buf[warp * 8 + lane] = c;
        __syncthreads();
        c = 0.f;
        for (int w0 = 0; w0 < nw; w0 += 16)
#pragma unroll
            for (int w = 0; w < 16; w += 4) c += buf[(w0 + w) * 8 + lane];
        c += __shfl_xor_sync(0xffffffffu, c, 8);
        c += __shfl_xor_sync(0xffffffffu, c, 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, c, i);
}

__device__ __forceinline__ float block_sum(float v, float* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (nw > 1) {
        if (lane == 0) buf[warp] = v;
        __syncthreads();
        v = lane < nw ? buf[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// A block of the row kernels holds one row: threads, at most, and the vectors
// of a thread (1, 2, 4 or 8).  256 threads with two or more blocks an SM keep
// more rows in flight than one block of 512.
constexpr int kNormThreads = 256;
void row_shape(int row_vec, int& kv, int& threads) {
    kv = 1;
    while (kv * kNormThreads < row_vec) kv *= 2;
    threads = (((row_vec + kv - 1) / kv) + 31) / 32 * 32;
}

constexpr int kNormGradThreads = 1024;       // of the norms' gradient, an SM
constexpr int kNormStageBytes = 216 * 1024;  // shared memory of an SM's gradient blocks
constexpr int kMaxCachedDevices = 64;

}  // namespace

bool row_kernels_fit(int H, int dtype) { return H <= 32 * 1024 / (dtype == 0 ? 2 : 4); }

// ------------------------------------------------------------- block norm
// For one token:  y = the block's output (given, or the combine's weighted sum
// of its K expert rows plus the shared output),
//   z = y rsqrt(mean y^2 + eps) w_post   (y without a norm after the block)
//   h = res_scale residual + gate z
//   n = h rsqrt(mean h^2 + eps) w_next   (the norm before the next block)
// One block per token, the row in registers as fp32 from the first load to
// the last store, so every output is rounded once; the K rows' vectors are all
// requested before the first is used.  2048 tokens of 3584 bf16, K = 8, shared
// output, both norms: 41 us, 191 MB (0.72 of the copy bandwidth); one token
// 2.7 us in a graph.  Without the combine, 4096 of 7168, gate and both norms:
// 63 us, 235 MB (0.58).
template <typename T, int kV, int kMaxK>
__global__ void __launch_bounds__(kNormThreads, kV <= 2 && kMaxK <= 8 ? 3 : 2) block_norm_kernel(BlockNormArgs a) {
    constexpr int N = Vec16<T>::N;
    constexpr bool kCombine = kMaxK > 0;
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int row_vec = a.H / N;
    const long long t = blockIdx.x;
    const long long base = t * row_vec;
    const int4* res = static_cast<const int4*>(a.residual);
    const int4* wpost = static_cast<const int4*>(a.w_post);
    const int4* wnext = static_cast<const int4*>(a.w_next);
    const int4* gate = static_cast<const int4*>(a.gate);
    const long long gbase = a.gate_mode == 2 ? base : 0;
    float y[kV][N];
    int4 rv[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        rv[j] = make_int4(0, 0, 0, 0);
        if (res && v < row_vec) rv[j] = res[base + v];
#pragma unroll
        for (int i = 0; i < N; ++i) y[j][i] = 0.f;
    }
    if constexpr (kCombine) {
        const int4* yp = static_cast<const int4*>(a.y);
        const int4* sh = static_cast<const int4*>(a.shared_out);
        int p[kMaxK];
        float w[kMaxK];
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
            p[k] = k < a.K ? __ldg(a.pos + t * a.K + k) : -1;
            w[k] = k < a.K ? __ldg(a.topk_w + t * a.K + k) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < row_vec) {
                int4 yv[kMaxK];
                int4 sv = make_int4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kMaxK; ++k)
                    if (p[k] >= 0) yv[k] = __ldcs(yp + (long long)p[k] * row_vec + v);
                if (sh) sv = __ldcs(sh + base + v);
#pragma unroll
                for (int k = 0; k < kMaxK; ++k) {
                    if (p[k] >= 0) {  // empty slot (per-token dynamic K): skipped
                        float f[N];
                        up<T>(yv[k], f);
#pragma unroll
                        for (int i = 0; i < N; ++i) y[j][i] += w[k] * f[i];
                    }
                }
                if (sh) {
                    float f[N];
                    up<T>(sv, f);
#pragma unroll
                    for (int i = 0; i < N; ++i) y[j][i] += f[i];
                }
                if (a.y_out) static_cast<int4*>(a.y_out)[base + v] = down<T>(y[j]);
            }
        }
    } else if (a.y) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < row_vec) up<T>(static_cast<const int4*>(a.y)[base + v], y[j]);
        }
    }
    float r = 1.f;
    if (wpost) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kV; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) s += y[j][i] * y[j][i];
        r = rsqrtf(block_sum(s, red[0]) / a.H + a.eps);
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < row_vec) {
            float f[N];
            if (wpost) {
                up<T>(__ldg(wpost + v), f);
#pragma unroll
                for (int i = 0; i < N; ++i) y[j][i] *= r * f[i];
            }
            if (gate) {
                up<T>(__ldg(gate + gbase + v), f);
#pragma unroll
                for (int i = 0; i < N; ++i) y[j][i] *= f[i];
            }
            up<T>(rv[j], f);
            if (res) {
#pragma unroll
                for (int i = 0; i < N; ++i) y[j][i] = fmaf(a.res_scale, f[i], y[j][i]);
            }
            if (a.h) static_cast<int4*>(a.h)[base + v] = down<T>(y[j]);
#pragma unroll
            for (int i = 0; i < N; ++i) s += y[j][i] * y[j][i];
        }
    }
    if (!wnext) return;
    r = rsqrtf(block_sum(s, red[1]) / a.H + a.eps);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < row_vec) {
            float f[N];
            up<T>(__ldg(wnext + v), f);
#pragma unroll
            for (int i = 0; i < N; ++i) y[j][i] *= r * f[i];
            static_cast<int4*>(a.n)[base + v] = down<T>(y[j]);
        }
    }
}

int launch_block_norm(const BlockNormArgs& a, cudaStream_t stream) {
    if (a.T == 0) return 0;
    int kv, threads;
    row_shape(a.H * (a.dtype == 0 ? 2 : 4) / 16, kv, threads);
    if (kv > 8) return -1;
    const dim3 g((unsigned)a.T), b(threads);
    cudaError_t e;
    auto go = [&](auto tag, auto kvc, auto kmax) -> cudaError_t {
        using E = typename std::remove_pointer<decltype(tag)>::type;
        return launch_kernel(block_norm_kernel<E, decltype(kvc)::value, decltype(kmax)::value>, g, b, 0, stream, a);
    };
    auto go_k = [&](auto tag, auto kvc) -> cudaError_t {
        if (!a.pos) return go(tag, kvc, std::integral_constant<int, 0>());
        if (a.K <= 2) return go(tag, kvc, std::integral_constant<int, 2>());
        if (a.K <= 8) return go(tag, kvc, std::integral_constant<int, 8>());
        return go(tag, kvc, std::integral_constant<int, 16>());
    };
    auto go_v = [&](auto tag) -> cudaError_t {
        if (kv == 1) return go_k(tag, std::integral_constant<int, 1>());
        if (kv == 2) return go_k(tag, std::integral_constant<int, 2>());
        if (kv == 4) return go_k(tag, std::integral_constant<int, 4>());
        return go_k(tag, std::integral_constant<int, 8>());
    };
    e = a.dtype == 0 ? go_v((__nv_bfloat16*)nullptr) : go_v((float*)nullptr);
    return launched(e);
}

// ---------------------------------------------------- block norm's gradient
// With rho_x = (mean x^2 + eps)^-1/2 and z, h, n as above:
//   d    = dh + rho_h (w_next dn - h rho_h^2 mean(w_next dn h))   (h's whole gradient)
//   dres = res_scale d;   dz = gate d;   dgate = d z (summed over the tokens for a channel gate)
//   dy   = rho_y (w_post dz - y rho_y^2 mean(w_post dz y))
//   dw_next = sum_t dn h rho_h;   dw_post = sum_t dz y rho_y
// The second mean is a linear function of d, so with
//   mean(w_post gate d y) = S(dh) + rho_h S(w_next dn) - rho_h^3 mean(w_next dn h) S(h),
//   S(x) = mean(w_post gate x y)
// six sums taken in one round give both means: one barrier per token.
// For a channel gate both dw_post and dgate are products of one column sum,
// A = sum_t d y rho_y (dw_post = gate A, dgate = w_post A).
// The kernel is bound by its instructions and their latency more than by
// memory (a row is 57 KB at 7168 bf16 with every input).  So it is laid out
// for 1024 threads an SM: a thread holds one vector's column sums (two in rows
// past 16 KB), and its values pass four at a time through few registers from
// shared memory, where cp.async has brought them two rows ahead (each thread
// copies its own vectors: no barrier).  Arithmetic is on pairs of floats
// (f32x2), the [H] vectors stay in shared memory, the product of w_post and a
// channel gate as fp32.  What a call has is fixed at compile time where it
// decides what is computed (kBlock: y; kGate: the gate's mode; kNext: w_next):
// tested in the loops it made 990 instructions of a vector's 300.  Persistent
// blocks take tokens block-stride; their column sums go to the workspace as
// one fp32 row per block and are added in block order by norm_wgrad_kernel:
// deterministic.  4096 tokens of 7168 bf16 with every part: 87 us, 352 MB (0.63
// of the copy bandwidth; issue slots 61 % used); 448 threads holding rows in
// registers took 131 us.

// Two floats in a register pair, and operations on both (each rounded as the
// scalar operation).
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_make(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_split(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_both(float a) { return f2_make(a, a); }
__device__ __forceinline__ float f2_sum(f2 v) {
    float a, b;
    f2_split(v, a, b);
    return a + b;
}

// Elements 4 q .. 4 q + 3 of a 16-byte vector.
__device__ __forceinline__ void quad(const int4* v, int q, f2 (&f)[2], const __nv_bfloat16*) {
    const int2 x = reinterpret_cast<const int2*>(v)[q];
    f[0] = f2_make(__int_as_float(x.x << 16), __int_as_float(x.x & 0xffff0000));
    f[1] = f2_make(__int_as_float(x.y << 16), __int_as_float(x.y & 0xffff0000));
}
__device__ __forceinline__ void quad(const int4* v, int q, f2 (&f)[2], const float*) {
    const float4 x = reinterpret_cast<const float4*>(v)[q];
    f[0] = f2_make(x.x, x.y);
    f[1] = f2_make(x.z, x.w);
}
__device__ __forceinline__ void put_quad(int4* v, int q, const f2 (&f)[2], const __nv_bfloat16*) {
    float x[4];
    f2_split(f[0], x[0], x[1]);
    f2_split(f[1], x[2], x[3]);
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    __stcs(reinterpret_cast<int2*>(v) + q,
           make_int2(*reinterpret_cast<const int*>(&a), *reinterpret_cast<const int*>(&b)));
}
__device__ __forceinline__ void put_quad(int4* v, int q, const f2 (&f)[2], const float*) {
    float x[4];
    f2_split(f[0], x[0], x[1]);
    f2_split(f[1], x[2], x[3]);
    __stcs(reinterpret_cast<float4*>(v) + q, make_float4(x[0], x[1], x[2], x[3]));
}

template <typename T, int kV, bool kBlock, int kGate, bool kNext>
struct NormGradShape {
    // the streams of a row and their places in a stage
    static constexpr int kDh = 0, kY = 1, kH = kY + kBlock, kDn = kH + kNext, kTokGate = kDn + kNext;
    static constexpr int kIn = kTokGate + (kGate == 2);
    // shared memory before the stages, in 16-byte vectors a vector of the row:
    // fp32 coefficients w_post * channel gate, then w_next (rows past 16 KB
    // have no room for them and read them from global memory)
    static constexpr bool kHeld = kV == 1;
    static constexpr int kCoef = kHeld && kBlock ? (int)(4 / sizeof(T)) : 0;
    static constexpr int kHead = kHeld ? kCoef + kNext : 0;
};

template <typename T, int kV, bool kBlock, int kGate, bool kNext>
__global__ void __launch_bounds__(kNormGradThreads) block_norm_grad_kernel(BlockNormGradArgs a, int stages) {
    using S = NormGradShape<T, kV, kBlock, kGate, kNext>;
    constexpr int N = Vec16<T>::N;
    constexpr int kQ = N / 4;
    extern __shared__ int4 smem[];  // [kHead + stages * kIn][kV][threads]
    __shared__ float red[2][32 * 8];
    pdl_launch_dependents();
    pdl_wait();
    const int row_vec = a.H / N;
    const int nt = blockDim.x, tid = threadIdx.x, stream = kV * nt;
    const bool post = kBlock && a.w_post != nullptr;
    const float inv_h = 1.f / a.H;
    const T* tag = nullptr;
    const f2 zero2 = f2_both(0.f);
    for (int i = tid; i < 2 * 32 * 8; i += nt)
        if ((i & 255) >= nt / 4) red[i >> 8][i & 255] = 0.f;  // warps the block has not: read by block_sum8
    float4* coef = reinterpret_cast<float4*>(smem);  // quad q of vector v at [q * stream + v]
    // Every other eight lanes take their two quads of a bf16 vector the other way
    // round, so that sixteen lanes' 8-byte reads, 16 bytes apart, meet all banks
    // once: quad k of a thread (the index of its sums) is quad k ^ swap of the
    // vector.  Where shared memory is what is waited for: with a gate per token,
    // and in rows past 16 KB (4096 x 7168, token gate: 111 us without, 104 us; 2048
    // x 16384: 145 us, 137 us); elsewhere the added address arithmetic costs more
    // (32768 x 2048: 158 us without, 164 us)
    const int swap = kQ == 2 && (kGate == 2 || kV == 2) ? (tid >> 3) & 1 : 0;
    int4* wnext = smem + S::kCoef * stream;
    int4* rows = smem + S::kHead * stream;
    const int stage_vec = S::kIn * stream;
    auto fetch = [&](long long t, int stage) {
        if (t < a.T) {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int v = tid + j * nt;
                if (v < row_vec) {
                    int4* dst = rows + stage * stage_vec + v;
                    const long long o = t * row_vec + v;
                    if (a.dh) cp_async16(dst + S::kDh * stream, static_cast<const int4*>(a.dh) + o);
                    if (kBlock) cp_async16(dst + S::kY * stream, static_cast<const int4*>(a.y) + o);
                    if (kNext) {
                        cp_async16(dst + S::kH * stream, static_cast<const int4*>(a.h) + o);
                        cp_async16(dst + S::kDn * stream, static_cast<const int4*>(a.dn) + o);
                    }
                    if (kGate == 2) cp_async16(dst + S::kTokGate * stream, static_cast<const int4*>(a.gate) + o);
                }
            }
        }
        cp_async_commit();
    };
    auto wait = [&]() {  // the oldest stage has landed
        if (stages == 3) cp_async_wait<2>();
        else if (stages == 2) cp_async_wait<1>();
        else cp_async_wait<0>();
    };
    // w_post * channel gate (1 where there is none) and w_next
    auto coef_of = [&](int v, int q, f2 (&c)[2]) {
        c[0] = c[1] = f2_both(1.f);
        if (post) quad(static_cast<const int4*>(a.w_post) + v, q, c, tag);
        if (kGate == 1) {
            f2 g[2];
            quad(static_cast<const int4*>(a.gate) + v, q, g, tag);
            c[0] = f2_mul(c[0], g[0]);
            c[1] = f2_mul(c[1], g[1]);
        }
    };
    auto get_coef = [&](int v, int q, f2 (&c)[2]) {
        if (S::kHeld) quad(reinterpret_cast<const int4*>(coef + q * stream + v), 0, c, (const float*)nullptr);
        else coef_of(v, q, c);
    };
    auto get_wnext = [&](int v, int q, f2 (&f)[2]) {
        quad((S::kHeld ? wnext : static_cast<const int4*>(a.w_next)) + v, q, f, tag);
    };
    for (int s = 0; s < stages - 1; ++s) fetch((long long)blockIdx.x + (long long)s * gridDim.x, s);
    f2 acc_next[kV][N / 2], acc_post[kV][N / 2];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = tid + j * nt;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) acc_next[j][i] = acc_post[j][i] = zero2;
        if (!a.dh)  // an absent dh is a row of zeros
            for (int s = 0; s < stages; ++s) rows[s * stage_vec + S::kDh * stream + v] = make_int4(0, 0, 0, 0);
        if (v < row_vec) {
            if (S::kHeld && kBlock) {
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    f2 c[2];
                    coef_of(v, q, c);
                    float4 x;
                    f2_split(c[0], x.x, x.y);
                    f2_split(c[1], x.z, x.w);
                    coef[q * stream + v] = x;
                }
            }
            if (S::kHeld && kNext) wnext[v] = __ldg(static_cast<const int4*>(a.w_next) + v);
        }
    }
    int stage = 0, phase = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x, phase ^= 1) {
        // the place of the row before this one takes the row `stages - 1` ahead
        fetch(t + (long long)(stages - 1) * gridDim.x, stage == 0 ? stages - 1 : stage - 1);
        wait();
        const int4* row = rows + stage * stage_vec;
        f2 p[6];
#pragma unroll
        for (int i = 0; i < 6; ++i) p[i] = zero2;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int v = tid + j * nt;
            if (v < row_vec) {
#pragma unroll
                for (int k = 0; k < kQ; ++k) {
                    const int q = k ^ swap;
                    f2 h[2], dn[2], c[2], f[2];
                    if (kNext) {
                        quad(row + S::kH * stream + v, q, h, tag);
                        quad(row + S::kDn * stream + v, q, dn, tag);
                        get_wnext(v, q, f);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            dn[i] = f2_mul(dn[i], f[i]);
                            p[0] = f2_fma(h[i], h[i], p[0]);
                            p[1] = f2_fma(dn[i], h[i], p[1]);
                        }
                    }
                    if (post) {
                        quad(row + S::kY * stream + v, q, f, tag);
                        get_coef(v, q, c);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            p[2] = f2_fma(f[i], f[i], p[2]);
                            c[i] = f2_mul(c[i], f[i]);
                        }
                        if (kGate == 2) {
                            quad(row + S::kTokGate * stream + v, q, f, tag);
                            c[0] = f2_mul(c[0], f[0]);
                            c[1] = f2_mul(c[1], f[1]);
                        }
                        quad(row + S::kDh * stream + v, q, f, tag);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            p[3] = f2_fma(c[i], f[i], p[3]);
                            if (kNext) {
                                p[4] = f2_fma(c[i], dn[i], p[4]);
                                p[5] = f2_fma(c[i], h[i], p[5]);
                            }
                        }
                    }
                }
            }
        }
        float s[8];
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = f2_sum(p[i]);
        s[6] = s[7] = 0.f;
        if (kNext || kBlock) block_sum8(s, red[phase]);
        const float rho_h = kNext ? rsqrtf(s[0] * inv_h + a.eps) : 0.f;
        const float mean_h = kNext ? s[1] * inv_h * rho_h * rho_h * rho_h : 0.f;  // h's coefficient in d
        const float rho_y = post ? rsqrtf(s[2] * inv_h + a.eps) : 1.f;
        const float mean_y =
            post ? (s[3] + rho_h * s[4] - mean_h * s[5]) * inv_h * rho_y * rho_y * rho_y : 0.f;
        const f2 rh = f2_both(rho_h), mh = f2_both(-mean_h), ry = f2_both(rho_y), my = f2_both(-mean_y);
        const f2 scale = f2_both(a.res_scale);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int v = tid + j * nt;
            if (v < row_vec) {
                const long long o = t * row_vec + v;
#pragma unroll
                for (int k = 0; k < kQ; ++k) {
                    const int q = k ^ swap;
                    f2 d[2], x[2], f[2], g[2];
                    quad(row + S::kDh * stream + v, q, d, tag);
                    if (kNext) {
                        quad(row + S::kH * stream + v, q, x, tag);
                        quad(row + S::kDn * stream + v, q, g, tag);
                        get_wnext(v, q, f);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            g[i] = f2_mul(g[i], rh);
                            acc_next[j][2 * k + i] = f2_fma(g[i], x[i], acc_next[j][2 * k + i]);
                            d[i] = f2_fma(f[i], g[i], d[i]);
                            d[i] = f2_fma(mh, x[i], d[i]);
                        }
                    }
                    if (a.dresidual) {
                        f[0] = f2_mul(d[0], scale);
                        f[1] = f2_mul(d[1], scale);
                        put_quad(static_cast<int4*>(a.dresidual) + o, q, f, tag);
                    }
                    if (kBlock) {
                        quad(row + S::kY * stream + v, q, x, tag);
                        get_coef(v, q, f);
                        if (kGate == 2) quad(row + S::kTokGate * stream + v, q, g, tag);
                        f2 dg[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            d[i] = f2_mul(d[i], ry);
                            if (kGate == 2) {
                                const f2 e = f2_mul(d[i], x[i]);  // d y rho_y
                                dg[i] = f2_mul(e, f[i]);
                                acc_post[j][2 * k + i] = f2_fma(g[i], e, acc_post[j][2 * k + i]);
                                d[i] = f2_mul(d[i], g[i]);
                            } else {
                                acc_post[j][2 * k + i] = f2_fma(d[i], x[i], acc_post[j][2 * k + i]);
                            }
                            f[i] = f2_mul(f[i], d[i]);
                            if (post) f[i] = f2_fma(my, x[i], f[i]);  // else not of y: it may be infinite or NaN
                        }
                        if (kGate == 2) put_quad(static_cast<int4*>(a.dgate) + o, q, dg, tag);
                        put_quad(static_cast<int4*>(a.dy) + o, q, f, tag);
                    }
                }
            }
        }
        stage = stage == stages - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    // one fp32 row per block: [gridDim.x][2][H]
    float* part = a.partials + (long long)blockIdx.x * 2 * a.H;
    auto put_sums = [&](float* dst, const f2* s) {
#pragma unroll
        for (int k = 0; k < kQ; ++k) {
            float4 x;
            f2_split(s[2 * k], x.x, x.y);
            f2_split(s[2 * k + 1], x.z, x.w);
            *reinterpret_cast<float4*>(dst + 4 * (k ^ swap)) = x;
        }
    };
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = tid + j * nt;
        if (v < row_vec) {
            if (kNext) put_sums(part + (long long)v * N, acc_next[j]);
            if (kBlock) put_sums(part + a.H + (long long)v * N, acc_post[j]);
        }
    }
}

// The blocks' column sums added in block order: a block takes 32 columns, its
// 128 groups of threads a run of rows each (all in flight at once), then the
// groups are added in order, eight at a time.  blockIdx.y 0: dw_next; 1:
// dw_post and, for a channel gate, dgate.
constexpr int kWgradGroups = 128, kWgradCols = 32;

template <typename T>
__global__ void __launch_bounds__(kWgradGroups * kWgradCols / 4) norm_wgrad_kernel(BlockNormGradArgs a, int n_parts) {
    constexpr int kLanes = kWgradCols / 4, kFold = 8;
    __shared__ float4 sum[kWgradGroups][kLanes];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const int c = blockIdx.x * kWgradCols + lane * 4;
    const bool post = blockIdx.y == 1, in = c < a.H;
    auto add = [](float4& s, const float4& v) {
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    };
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
        const float* p = a.partials + (post ? a.H : 0) + c;
        const int per = (n_parts + kWgradGroups - 1) / kWgradGroups;
        const int end = min(n_parts, (grp + 1) * per);
#pragma unroll 8
        for (int r = grp * per; r < end; ++r)
            add(s, __ldcs(reinterpret_cast<const float4*>(p + (long long)r * 2 * a.H)));
    }
    sum[grp][lane] = s;
    __syncthreads();
    if (grp < kWgradGroups / kFold) {
        s = sum[grp * kFold][lane];
#pragma unroll
        for (int g = 1; g < kFold; ++g) add(s, sum[grp * kFold + g][lane]);
    }
    __syncthreads();
    if (grp < kWgradGroups / kFold) sum[grp][lane] = s;
    __syncthreads();
    if (grp != 0 || !in) return;
#pragma unroll
    for (int g = 1; g < kWgradGroups / kFold; ++g) add(s, sum[g][lane]);
    if (!post) {
        if (a.dw_next) *reinterpret_cast<float4*>(a.dw_next + c) = s;
        return;
    }
    const float f[4] = {s.x, s.y, s.z, s.w};
    // without tokens the sums are zero whatever the weights are
    const T* g = n_parts && a.gate_mode == 1 ? static_cast<const T*>(a.gate) : nullptr;
    const T* w = n_parts ? static_cast<const T*>(a.w_post) : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (a.dw_post) a.dw_post[c + i] = g ? Elt<T>::to_f(g[c + i]) * f[i] : f[i];
        if (a.gate_mode == 1 && a.dgate)
            static_cast<float*>(a.dgate)[c + i] = w ? Elt<T>::to_f(w[c + i]) * f[i] : f[i];
    }
}

namespace {
// One vector a thread, two in rows of more than 1024 vectors.
void norm_grad_shape(int H, int dtype, int& kv, int& threads) {
    const int row_vec = H * (dtype == 0 ? 2 : 4) / 16;
    kv = row_vec <= kNormGradThreads ? 1 : 2;
    threads = (((row_vec + kv - 1) / kv) + 31) / 32 * 32;
}
}  // namespace

// Blocks of the gradient kernel: 1024 threads per SM, so that short rows are
// not left waiting for one another, at most 16 blocks.
int norm_grad_blocks(int T, int H, int dtype, int num_sms) {
    int kv, threads;
    norm_grad_shape(H, dtype, kv, threads);
    int per_sm = kNormGradThreads / threads;
    if (per_sm > 16) per_sm = 16;
    const long long most = (long long)num_sms * per_sm;
    return T < most ? T : (int)most;
}

namespace {
template <typename T, int kV, bool kBlock, int kGate, bool kNext>
cudaError_t launch_norm_grad_rows(const BlockNormGradArgs& a, const DeviceInfo& d, int blocks, int threads,
                                  cudaStream_t stream) {
    auto kern = block_norm_grad_kernel<T, kV, kBlock, kGate, kNext>;
    static std::atomic<bool> raised[kMaxCachedDevices];  // per instantiation: the shared-memory limit
    if (!raised[d.device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormStageBytes);
        if (e != cudaSuccess) return e;
        raised[d.device].store(true, std::memory_order_release);
    }
    // three rows at once, fewer where the rows are so long that they do not fit
    // (the blocks of an SM share it)
    using S = NormGradShape<T, kV, kBlock, kGate, kNext>;
    const int vecs = kV * threads * 16;
    int stages = (kNormStageBytes / (kNormGradThreads / threads) - S::kHead * vecs) / (S::kIn * vecs);
    if (stages > 3) stages = 3;
    if (stages < 1) return cudaErrorInvalidValue;
    return launch_kernel(kern, dim3(blocks), dim3(threads), (S::kHead + stages * S::kIn) * vecs, stream, a,
                         stages);
}

template <typename T, int kV>
cudaError_t launch_norm_grad_form(const BlockNormGradArgs& a, const DeviceInfo& d, int blocks, int threads,
                                  cudaStream_t s) {
    if (!a.y) {
        if (a.w_next) return launch_norm_grad_rows<T, kV, false, 0, true>(a, d, blocks, threads, s);
        return launch_norm_grad_rows<T, kV, false, 0, false>(a, d, blocks, threads, s);
    }
    auto gate = [&](auto g) {
        constexpr int kGate = decltype(g)::value;
        if (a.w_next) return launch_norm_grad_rows<T, kV, true, kGate, true>(a, d, blocks, threads, s);
        return launch_norm_grad_rows<T, kV, true, kGate, false>(a, d, blocks, threads, s);
    };
    if (a.gate_mode == 0) return gate(std::integral_constant<int, 0>());
    if (a.gate_mode == 1) return gate(std::integral_constant<int, 1>());
    return gate(std::integral_constant<int, 2>());
}
}  // namespace

int launch_block_norm_grad(const BlockNormGradArgs& a, cudaStream_t stream) {
    DeviceInfo d;
    int rc = current_device(&d);
    if (rc != 0) return rc;
    if (!row_kernels_fit(a.H, a.dtype)) return -1;
    int kv, threads;
    norm_grad_shape(a.H, a.dtype, kv, threads);
    const int blocks = norm_grad_blocks(a.T, a.H, a.dtype, d.num_sms);
    if (blocks > 0) {
        using bf = __nv_bfloat16;
        const cudaError_t e =
            a.dtype == 0 ? (kv == 1 ? launch_norm_grad_form<bf, 1>(a, d, blocks, threads, stream)
                                    : launch_norm_grad_form<bf, 2>(a, d, blocks, threads, stream))
                         : (kv == 1 ? launch_norm_grad_form<float, 1>(a, d, blocks, threads, stream)
                                    : launch_norm_grad_form<float, 2>(a, d, blocks, threads, stream));
        if ((rc = launched(e)) != 0) return rc;
    }
    const bool post = a.dw_post || (a.dgate && a.gate_mode == 1);
    if (!a.dw_next && !post) return 0;
    const dim3 g((a.H + kWgradCols - 1) / kWgradCols, post ? 2 : 1), b(kWgradGroups * kWgradCols / 4);
    return launched(a.dtype == 0
                        ? launch_kernel(norm_wgrad_kernel<__nv_bfloat16>, g, b, 0, stream, a, blocks)
                        : launch_kernel(norm_wgrad_kernel<float>, g, b, 0, stream, a, blocks));
}

// ------------------------------------------------------ combine's gradient
// dy_perm[pos(t,k)] = w(t,k) dout[t];  dw(t,k) = <dout[t], y_perm[pos(t,k)]>.
// One block per token: dout's row is read once into registers and meets the K
// rows it scales and is dotted with.  The blocks past the tokens zero the
// padding rows (the weight gradients multiply them).  4096 tokens of 7168
// bf16, K = 8: 177 us (a single call 184 us), 1.0 GB (0.87 of the copy
// bandwidth).
template <typename T, int kV, int kMaxK>
__global__ void __launch_bounds__(kNormThreads, 2) combine_grad_kernel(CombineGradArgs a) {
    constexpr int N = Vec16<T>::N;
    __shared__ float red[kMaxK][32];
    pdl_launch_dependents();
    pdl_wait();
    const int row_vec = a.H / N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int4* dy = static_cast<int4*>(a.dy_perm);
    if (blockIdx.x >= (unsigned)a.T) {
        // pad_slots (at most 32) slots at a time, a padding row by the whole block
        const int P = a.scalars[0];
        const long long step = (long long)(gridDim.x - a.T) * a.pad_slots;
        for (long long p0 = (long long)(blockIdx.x - a.T) * a.pad_slots; p0 < P; p0 += step) {
            const bool pad = lane < a.pad_slots && p0 + lane < P && __ldg(a.sorted_ids + p0 + lane) < 0;
            for (unsigned m = __ballot_sync(0xffffffffu, pad); m; m &= m - 1) {
                int4* row = dy + (p0 + __ffs(m) - 1) * row_vec;
                for (int v = threadIdx.x; v < row_vec; v += blockDim.x) __stcs(row + v, make_int4(0, 0, 0, 0));
            }
        }
        return;
    }
    const long long t = blockIdx.x;
    int4 dv[kV];  // dout's row, as it came: unpacked for each of the K rows it meets
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        dv[j] = make_int4(0, 0, 0, 0);
        if (v < row_vec) dv[j] = __ldcs(static_cast<const int4*>(a.dout) + t * row_vec + v);
    }
    // kB rows requested before the first is used (16 vectors a thread: 115 KB an
    // SM): dy_perm may be y_perm, so no load can move above an earlier row's
    // store by itself
    constexpr int kB = kMaxK < 16 / kV ? kMaxK : 16 / kV;
    float dot[kMaxK];
#pragma unroll
    for (int k0 = 0; k0 < kMaxK; k0 += kB) {
        int p[kB];
        float w[kB];
        int4 yv[kB][kV];
#pragma unroll
        for (int b = 0; b < kB; ++b) {
            p[b] = k0 + b < a.K ? __ldg(a.pos + t * a.K + k0 + b) : -1;
            w[b] = k0 + b < a.K ? __ldg(a.topk_w + t * a.K + k0 + b) : 0.f;
        }
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int v = threadIdx.x + j * blockDim.x;
                if (p[b] >= 0 && v < row_vec)
                    yv[b][j] = __ldcs(static_cast<const int4*>(a.y_perm) + (long long)p[b] * row_vec + v);
            }
#pragma unroll
        for (int b = 0; b < kB; ++b) {
            dot[k0 + b] = 0.f;
            if (p[b] >= 0) {
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const int v = threadIdx.x + j * blockDim.x;
                    if (v < row_vec) {
                        float f[N], d[N];
                        up<T>(yv[b][j], f);
                        up<T>(dv[j], d);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            dot[k0 + b] += d[i] * f[i];
                            f[i] = w[b] * d[i];
                        }
                        __stcs(dy + (long long)p[b] * row_vec + v, down<T>(f));
                    }
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
        if (lane == 0) red[k][warp] = dot[k];
    }
    __syncthreads();
    for (int k = warp; k < a.K; k += nw) {
        float s = lane < nw ? red[k][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) a.dw[t * a.K + k] = s;
    }
}

int launch_combine_grad(const CombineGradArgs& args, cudaStream_t stream) {
    DeviceInfo d;
    int rc = current_device(&d);
    if (rc != 0) return rc;
    int kv, threads;
    row_shape(args.H * (args.dtype == 0 ? 2 : 4) / 16, kv, threads);
    if (kv > 8) return -1;
    // few slots a block where that spreads a few padding rows over the SMs
    CombineGradArgs a = args;
    a.pad_slots = a.P_max < 32LL * d.num_sms ? 4 : 32;
    long long pad_blocks = (a.P_max + a.pad_slots - 1) / a.pad_slots;
    if (pad_blocks > 4LL * d.num_sms) pad_blocks = 4LL * d.num_sms;
    if (a.T + pad_blocks > INT_MAX) return -1;
    const dim3 g((unsigned)(a.T + pad_blocks)), b(threads);
    auto go = [&](auto tag, auto kvc, auto kmax) -> cudaError_t {
        using E = typename std::remove_pointer<decltype(tag)>::type;
        return launch_kernel(combine_grad_kernel<E, decltype(kvc)::value, decltype(kmax)::value>, g, b, 0, stream, a);
    };
    auto go_k = [&](auto tag, auto kvc) -> cudaError_t {
        if (a.K <= 2) return go(tag, kvc, std::integral_constant<int, 2>());
        if (a.K <= 8) return go(tag, kvc, std::integral_constant<int, 8>());
        return go(tag, kvc, std::integral_constant<int, 16>());
    };
    auto go_v = [&](auto tag) -> cudaError_t {
        if (kv == 1) return go_k(tag, std::integral_constant<int, 1>());
        if (kv == 2) return go_k(tag, std::integral_constant<int, 2>());
        if (kv == 4) return go_k(tag, std::integral_constant<int, 4>());
        return go_k(tag, std::integral_constant<int, 8>());
    };
    return launched(a.dtype == 0 ? go_v((__nv_bfloat16*)nullptr) : go_v((float*)nullptr));
}

// --------------------------------------------------------- gate's gradient
// One warp per token; lane j < K holds slot j's expert, logit and weight
// gradient.  With w the gate weights, p the full softmax, s the sigmoid:
//   softmax, renormalised: dl_i = w_i (dw_i - sum_j w_j dw_j) on the selected
//   softmax over all E:    dl_e = p_e (dw_e [e selected] - sum_j p_j dw_j)
//   sigmoid, renormalised: dl_i = w_i (1 - s_i) (dw_i - sum_j w_j dw_j)
//   sigmoid:               dl_i = s_i (1 - s_i) dw_i
// 1 - s is taken as the sigmoid of -l, so it keeps its digits near s = 1.
// The row is zeroed (or given the full softmax's share), then the selected
// entries are written; a repeated expert's shares are added first.  Bound by
// latency: 2048 tokens x 256 experts, K = 8, in a graph: 2.6 us, 2.3 MB on the
// selected logits; the full softmax, which passes over the row three times, 4.9 us.
__global__ void __launch_bounds__(256) route_grad_kernel(int T, int E, int K, int score_fn, int renorm,
                                                         const float* __restrict__ logits,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ dw, float* __restrict__ dlogits) {
    pdl_launch_dependents();
    pdl_wait();
    const long long t = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (t >= T) return;
    const float* l = logits + t * E;
    float* out = dlogits + t * E;
    auto wsum = [](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    auto wmax = [](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    };
    const int id = lane < K ? ids[t * K + lane] : -1;
    const bool on = id >= 0 && id < E;  // an empty slot has no gradient
    const float li = on ? l[id] : 0.f;
    const float di = on ? dw[t * K + lane] : 0.f;
    const bool full = score_fn == 0 && !renorm;
    float g;
    if (score_fn == 0) {
        float m = -INFINITY, den;
        if (full) {
            for (int e = lane; e < E; e += 32) m = fmaxf(m, l[e]);
            m = wmax(m);
            den = 0.f;
            for (int e = lane; e < E; e += 32) den += expf(l[e] - m);
            den = wsum(den);
        } else {
            m = wmax(on ? li : -INFINITY);
            den = wsum(on ? expf(li - m) : 0.f);
        }
        const float w = on ? expf(li - m) / den : 0.f;
        const float mean = wsum(w * di);
        g = full ? w * di : w * (di - mean);
        for (int e = lane; e < E; e += 32) out[e] = full ? -(expf(l[e] - m) / den) * mean : 0.f;
        if (full) {
            // the selected entries: their share of the row plus their own (shares of a repeated expert added below)
            float own = 0.f;
            for (int j = 0; j < K; ++j) {
                const int ij = __shfl_sync(0xffffffffu, on ? id : -1, j);
                const float gj = __shfl_sync(0xffffffffu, g, j);
                if (ij == id) own += gj;
            }
            __syncwarp();
            if (on) out[id] = own - w * mean;
            return;
        }
    } else {
        const float s = on ? 1.f / (1.f + expf(-li)) : 0.f;
        const float c = 1.f / (1.f + expf(li));  // 1 - s
        if (renorm) {
            const float den = wsum(s);
            const float w = on ? s / den : 0.f;
            g = w * c * (di - wsum(w * di));
        } else {
            g = s * c * di;
        }
        for (int e = lane; e < E; e += 32) out[e] = 0.f;
    }
    float own = 0.f;
    for (int j = 0; j < K; ++j) {
        const int ij = __shfl_sync(0xffffffffu, on ? id : -1, j);
        const float gj = __shfl_sync(0xffffffffu, g, j);
        if (ij == id) own += gj;
    }
    __syncwarp();  // the zeros are written before the selected entries
    if (on) out[id] = own;
}

int launch_route_grad(int T, int E, int K, int score_fn, int renorm, const float* logits, const int32_t* ids,
                      const float* dw, float* dlogits, cudaStream_t stream) {
    const int warps = 4;
    return launched(launch_kernel(route_grad_kernel, dim3((unsigned)((T + warps - 1) / warps)), dim3(32 * warps), 0,
                                  stream, T, E, K, score_fn, renorm, logits, ids, dw, dlogits));
}

}  // namespace moe

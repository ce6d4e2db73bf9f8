// AdamW over many tensors at once, with the gradient norm and its clipping.
//
//   N = sqrt(sum g^2) over every tensor; k = min(1, max_norm / N)
//   m = b1 m + (1 - b1) k g;  v = b2 v + (1 - b2) (k g)^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Two launches: the norm (every gradient once, and a CTA that advances the step;
// without clipping that one alone) and the update.  The list of tensors travels in the
// kernel's parameters (one launch for up to kAdamCap tensors), so nothing has
// to be copied to the device when gradients move from step to step.
//
// States are FP32, or 8 bits: E4M3 codes with one FP32 scale for 256 values
// (the largest magnitude of the 256 at the format's largest value, 448).  The
// second moment is kept as its root, which is what the update divides by: the
// root of a value spans half its octaves, so the codes' 17 octaves cover 35 of
// v, and a root that is not zero never rounds to zero (the divisor of a value
// whose gradients are small next to its neighbours' would lose its meaning).
// A block below 2^-100 is stored as zeros.  The codes are rounded once per
// step; the step itself uses the new moments in FP32.
//
// Bound by bandwidth: 30 bytes a value with 32-bit states, an FP32 gradient, a
// BF16 parameter and its FP32 master (562M values: the update 2.44 ms, 6.9 TB/s;
// the norm's pass over the gradients 0.34 ms, 6.6 TB/s), 16 with 8-bit states and
// BF16 gradients (317M values: 0.88 ms, 5.7 TB/s, as much held by the
// conversions and roots as by memory; the norm 0.13 ms).  A warp takes 256
// consecutive values (an 8-bit block), a lane four and four, so that every array
// is read and written in whole 128-byte lines, and issues every load first.
#include <algorithm>

#include <cuda_fp8.h>

#include "kernels.cuh"
#include "twosum.cuh"

namespace lrs {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                             // values a scale stands for, values of a warp
constexpr int kAdamChunk = kAdamBlock * kAdamThreads / 32;  // values of a CTA at a time
constexpr int kAdamNormCtas = 8;                            // CTAs per SM of the norm
constexpr float kFp8Max = 448.f, kFp8Inv = 1.f / 448.f;
constexpr float kFp8Tiny = 0.001953125f;                    // 2^-9, the smallest E4M3 value above 0
constexpr float kAdamSmall = 7.888609052210118e-31f;        // 2^-100

// The list of one launch, in the kernel's parameters.
template <int CAP>
struct AdamList {
    AdamTensor t[CAP];
    int first[CAP + 1];   // first chunk of each tensor; [count]: the chunks in all
    int count;
};

// The tensor of chunk c: the last one that starts at or before it.
template <int CAP>
__device__ __forceinline__ int adam_find(const AdamList<CAP>& l, int c) {
    int lo = 0, hi = l.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Four values from i on of an array of n; FULL: all four are inside it (else
// zeros past its end, and nothing is stored there).
template <bool FULL>
__device__ __forceinline__ void load_f32(const float* p, long long i, long long n, float (&v)[4]) {
    if (FULL) {
        const float4 q = *reinterpret_cast<const float4*>(p + i);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < n ? p[i + k] : 0.f;
    }
}
template <bool FULL>
__device__ __forceinline__ void store_f32(float* p, long long i, long long n, const float (&v)[4]) {
    if (FULL) {
        *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[i + k] = v[k];
    }
}
template <bool FULL>
__device__ __forceinline__ void load_bf16(const uint16_t* p, long long i, long long n, float (&v)[4]) {
    if (FULL) {
        const uint2 q = *reinterpret_cast<const uint2*>(p + i);
        const float2 a = bf2_to_f2(q.x), b = bf2_to_f2(q.y);
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < n ? __uint_as_float((uint32_t)p[i + k] << 16) : 0.f;
    }
}
template <bool FULL>
__device__ __forceinline__ void store_bf16(uint16_t* p, long long i, long long n, const float (&v)[4]) {
    const uint32_t w[2] = {f2_to_bf2(v[0], v[1]), f2_to_bf2(v[2], v[3])};
    if (FULL) {
        *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[i + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
    }
}
template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, long long i, long long n) {
    if (FULL) return *reinterpret_cast<const uint32_t*>(p + i);
    uint32_t q = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < n) q |= (uint32_t)p[i + k] << (8 * k);
    return q;
}
__device__ __forceinline__ void decode(uint32_t q, float s, float (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> (8 * k)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[k] = f.x * s;
        v[k + 1] = f.y * s;
    }
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* p, long long i, long long n, const float (&v)[4]) {
    const uint32_t q = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3) |
                       (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3) << 16;
    if (FULL) {
        *reinterpret_cast<uint32_t*>(p + i) = q;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[i + k] = (uint8_t)(q >> (8 * k));
    }
}

// Sum over the CTA in a fixed order; the result in every thread.
__device__ __forceinline__ TwoSum cta_sum(TwoSum v, float2* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(v.hi, v.lo);
    __syncthreads();
    TwoSum s;
#pragma unroll
    for (int w = 0; w < kAdamThreads / 32; ++w) s.add(red[w].x, red[w].y);
    return s;
}

// Squares of eight BF16 or four FP32 values (SCALED: times 2^-96 each), added to q.
constexpr float kAdamDown = 1.262177448e-29f, kAdamUp = 7.922816251e28f;   // 2^-96, 2^96
template <bool SCALED>
__device__ __forceinline__ void squares(const uint4 v, bool bf16, float& q) {
    auto add = [&](float x) {
        if (SCALED) x *= kAdamDown;
        q = fmaf(x, x, q);
    };
    if (bf16) {
        const float2 a = bf2_to_f2(v.x), b = bf2_to_f2(v.y), c = bf2_to_f2(v.z), d = bf2_to_f2(v.w);
        add(a.x); add(a.y); add(b.x); add(b.y);
        add(c.x); add(c.y); add(d.x); add(d.y);
    } else {
        add(__uint_as_float(v.x)); add(__uint_as_float(v.y)); add(__uint_as_float(v.z)); add(__uint_as_float(v.w));
    }
}
// A sum of squares whose N is in range though its squares are not: up to 32
// squares at a time are added in FP32; a sum of them from 2^80 on (below it 2^40
// values do not overflow) is formed again 2^-192 times as large and kept apart.
// NaN and infinities go there too.
constexpr float kAdamBig = 1.208925820e24f;   // 2^80
struct SquareSum {
    TwoSum mid, big;
};
// N sixteen-byte groups p[0], p[kAdamThreads], ... (x: loaded) added to a thread's
// sum.  Those out of range are read again and `big` is in shared memory: held in
// registers, they cost a CTA an SM (562M FP32 gradients 340 -> 350 us).
template <int N>
__device__ __forceinline__ void add_squares(const uint4* x, const uint4* p, bool bf16, TwoSum& mid, TwoSum& big) {
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) squares<false>(x[k], bf16, q);
    if (q < kAdamBig) {
        mid.add(q);
    } else {
        q = 0.f;
#pragma unroll 1
        for (int k = 0; k < N; ++k) squares<true>(__ldg(p + k * kAdamThreads), bf16, q);
        big.add(q);
    }
}
__device__ __forceinline__ void add_square(float x, TwoSum& mid, TwoSum& big) {
    if (x * x < kAdamBig) {
        mid.add(x * x);
    } else {
        x *= kAdamDown;
        big.add(x * x);
    }
}
// Sum over the CTA, in every thread; `big` is looked at where any thread has some.
__device__ __forceinline__ SquareSum cta_sum(const SquareSum& v, float2* red) {
    SquareSum s;
    s.mid = cta_sum(v.mid, red);
    if (__syncthreads_or(v.big.hi != 0.f)) s.big = cta_sum(v.big, red);
    return s;
}
// First launch of a step: sums of squares of the gradients, one partial sum a
// CTA, in a fixed order.  A chain of 32 squares loses at most 2^-19 of its value
// and the sums of the chains, in two floats, nothing: N is within 2^-19.  The last
// CTA advances the step and forms its bias corrections, 1 - b^t = -expm1(t log b).
template <int CAP>
__global__ void __launch_bounds__(kAdamThreads) adamw_norm_kernel(const __grid_constant__ AdamList<CAP> l,
                                                                  const AdamArgs a) {
    __shared__ float2 red[kAdamThreads / 32];
    pdl_trigger();
    pdl_wait();
    int ctas = (int)gridDim.x;
    if (a.advance) {
        --ctas;
        if ((int)blockIdx.x == ctas) {
            const int t = *a.step + 1;
            __syncthreads();
            if (threadIdx.x == 0) *a.step = t;
            if (threadIdx.x == 0 || threadIdx.x == 32) {
                const int k = threadIdx.x / 32;
                a.bias[k] = -1.f / expm1f((float)t * (k == 0 ? a.log_b1 : a.log_b2));
            }
            return;
        }
    }
    // groups of chunks, the CTAs in turns (runs of their own leave each CTA
    // streaming from a far place of its own, which is slower)
    // eight loads in flight a thread (317M BF16 gradients: 4 loads 148 us, 8 loads
    // 126; 562M FP32 ones 358 and 340); their squares enter the pair of floats in two parts of four, so that
    // the plain FP32 sums stay short
    constexpr int kUnroll = 8;
    const int chunks = l.first[l.count];
    __shared__ TwoSum bigs[kAdamThreads];
    TwoSum& big = bigs[threadIdx.x];
    big = TwoSum();
    TwoSum sum;
    for (int c0 = (int)blockIdx.x * a.norm_group; c0 < chunks; c0 += ctas * a.norm_group) {
        const int c1 = min(c0 + a.norm_group, chunks);
        int c = c0;
        for (int i = adam_find(l, c); c < c1; ++i) {
            // the group's part of tensor i, in units of 16 bytes and a rest
            const int to = min(c1, l.first[i + 1]);
            const bool bf = l.t[i].grad_dtype == LRS_GRAD_BF16;
            const int per = bf ? 8 : 4;
            const long long e0 = (long long)(c - l.first[i]) * kAdamChunk;
            const int n = (int)min((long long)(to - c) * kAdamChunk, (long long)l.t[i].n - e0), nv = n / per;
            const uint4* g = static_cast<const uint4*>(l.t[i].grad) + e0 / per;
            int v = threadIdx.x;
            for (; v + (kUnroll - 1) * kAdamThreads < nv; v += kUnroll * kAdamThreads) {
                uint4 x[kUnroll];
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) x[k] = __ldg(g + v + k * kAdamThreads);
#pragma unroll
                for (int h = 0; h < kUnroll; h += 4) add_squares<4>(x + h, g + v + h * kAdamThreads, bf, sum, big);
            }
            for (; v < nv; v += kAdamThreads) {
                const uint4 x = __ldg(g + v);
                add_squares<1>(&x, g + v, bf, sum, big);
            }
            const int e = nv * per + (int)threadIdx.x;
            if (e < n) {
                const float x = bf ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(g)[e] << 16)
                                   : reinterpret_cast<const float*>(g)[e];
                add_square(x, sum, big);
            }
            c = to;
        }
    }
    SquareSum s;
    s.mid = sum;
    s.big = big;
    s = cta_sum(s, red);
    if (threadIdx.x == 0)
        a.partial[a.partial0 + blockIdx.x] = make_float4(s.mid.hi, s.mid.lo, s.big.hi, s.big.lo);
}

// The step's scalars.
struct AdamScalars {
    float clip, lr, ibc1, root_ibc2, b1, c1, b2, c2, eps;
};

// 256 consecutive values of one tensor, by one warp.
template <bool Q8, bool GRAD_BF16, bool FULL>
__device__ __forceinline__ void adam_block(const AdamTensor& t, long long b0, int lane, const AdamScalars& a) {
    const long long n = t.n;
    const bool master = t.master != nullptr;
    float* p32 = master ? t.master : static_cast<float*>(t.param);
    float p[2][4], g[2][4], m[2][4], v[2][4];
    float ms = 0.f, vs = 0.f;
    uint32_t mc[2], vc[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const long long e = b0 + 128 * k + 4 * lane;
        if (GRAD_BF16)
            load_bf16<FULL>(static_cast<const uint16_t*>(t.grad), e, n, g[k]);
        else
            load_f32<FULL>(static_cast<const float*>(t.grad), e, n, g[k]);
        load_f32<FULL>(p32, e, n, p[k]);
        if (Q8) {
            mc[k] = load_codes<FULL>(static_cast<const uint8_t*>(t.m), e, n);
            vc[k] = load_codes<FULL>(static_cast<const uint8_t*>(t.v), e, n);
        } else {
            load_f32<FULL>(static_cast<const float*>(t.m), e, n, m[k]);
            load_f32<FULL>(static_cast<const float*>(t.v), e, n, v[k]);
        }
    }
    if (Q8) {
        ms = t.m_scale[b0 / kAdamBlock];
        vs = t.v_scale[b0 / kAdamBlock];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            decode(mc[k], ms, m[k]);
            decode(vc[k], vs, v[k]);
        }
    }
    const float keep = 1.f - a.lr * t.weight_decay;
    float root[2][4];
    uint32_t mtop = 0u, vtop = 0u;   // magnitudes as integers: their order is the values', NaN above all
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float gg = g[k][j] * a.clip;
            const float vv = Q8 ? v[k][j] * v[k][j] : v[k][j];
            // each product rounded by itself, as written above
            m[k][j] = __fadd_rn(__fmul_rn(m[k][j], a.b1), __fmul_rn(gg, a.c1));
            v[k][j] = __fadd_rn(__fmul_rn(vv, a.b2), __fmul_rn(__fmul_rn(gg, gg), a.c2));
            // one root serves the step and the state: correctly rounded where it
            // is stored (a code next to a tie follows its last bit), from the SFU
            // like the quotient otherwise, within 2^-22 (the step is a small part of
            // p; both correctly rounded: one small block 9.8 -> 11.8 us).  v may be
            // below 2^-126: a root of 0 would leave eps alone to divide by
            root[k][j] = Q8 ? __fsqrt_rn(v[k][j]) : sqrt_approx_full(v[k][j]);
            const float step = __fdividef(m[k][j] * a.ibc1, fmaf(root[k][j], a.root_ibc2, a.eps));
            p[k][j] = fmaf(-a.lr, step, p[k][j] * keep);
            if (Q8) {
                mtop = max(mtop, __float_as_uint(fabsf(m[k][j])));
                vtop = max(vtop, __float_as_uint(root[k][j]));
            }
        }
    }
    if (Q8) {
        const float mt = __uint_as_float(__reduce_max_sync(0xffffffffu, mtop));
        const float vt = __uint_as_float(__reduce_max_sync(0xffffffffu, vtop));
        // one reciprocal a block and products with constants
        const float mi = mt >= kAdamSmall ? __frcp_rn(mt) * kFp8Max : 0.f;
        const float vi = vt >= kAdamSmall ? __frcp_rn(vt) * kFp8Max : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[k][j] *= mi;
                const float r = root[k][j] * vi;
                v[k][j] = r > 0.f ? fmaxf(r, kFp8Tiny) : r;
            }
        if (lane == 0) {
            t.m_scale[b0 / kAdamBlock] = mt >= kAdamSmall ? mt * kFp8Inv : 0.f;
            t.v_scale[b0 / kAdamBlock] = vt >= kAdamSmall ? vt * kFp8Inv : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const long long e = b0 + 128 * k + 4 * lane;
        store_f32<FULL>(p32, e, n, p[k]);
        if (master) store_bf16<FULL>(static_cast<uint16_t*>(t.param), e, n, p[k]);
        if (Q8) {
            store_codes<FULL>(static_cast<uint8_t*>(t.m), e, n, m[k]);
            store_codes<FULL>(static_cast<uint8_t*>(t.v), e, n, v[k]);
        } else {
            store_f32<FULL>(static_cast<float*>(t.m), e, n, m[k]);
            store_f32<FULL>(static_cast<float*>(t.v), e, n, v[k]);
        }
    }
}
template <bool Q8, bool GRAD_BF16>
__device__ __forceinline__ void adam_block_any(const AdamTensor& t, long long b0, int lane, const AdamScalars& a) {
    if (b0 + kAdamBlock <= t.n)
        adam_block<Q8, GRAD_BF16, true>(t, b0, lane, a);
    else
        adam_block<Q8, GRAD_BF16, false>(t, b0, lane, a);
}

template <int CAP>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_update_kernel(const __grid_constant__ AdamList<CAP> l,
                                                                       const AdamArgs a) {
    __shared__ float2 red[kAdamThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    pdl_wait();
    AdamScalars sc;
    sc.clip = 1.f;
    if (a.max_norm > 0.f) {
        SquareSum s;
        for (int i = threadIdx.x; i < a.partials; i += kAdamThreads) {
            const float4 q = __ldcg(a.partial + i);
            s.mid.add(q.x, q.y);
            s.big.add(q.z, q.w);
        }
        s = cta_sum(s, red);
        const float norm = s.big.hi == 0.f ? sqrtf(s.mid.value())
                                           : sqrtf(s.big.value() + s.mid.value() * kAdamDown * kAdamDown) * kAdamUp;
        const bool skip = !(norm <= 3.4028234e38f);
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.advance) {
            *a.norm = norm;
            if (skip) *a.step -= 1;   // no other CTA of a skipped step reads it
        }
        if (skip) return;
        sc.clip = norm > a.max_norm ? a.max_norm / norm : 1.f;
    }
    sc.lr = __ldg(a.lr);
    sc.ibc1 = __ldcg(a.bias);
    sc.root_ibc2 = sqrtf(__ldcg(a.bias + 1));
    sc.b1 = a.b1;
    sc.c1 = a.c1;
    sc.b2 = a.b2;
    sc.c2 = a.c2;
    sc.eps = a.eps;
    for (int c = (int)blockIdx.x; c < l.first[l.count]; c += (int)gridDim.x) {
        const int i = adam_find(l, c);
        const AdamTensor& t = l.t[i];
        const long long b0 = (long long)(c - l.first[i]) * kAdamChunk + warp * kAdamBlock;
        if (b0 >= t.n) continue;
        const bool bf = t.grad_dtype == LRS_GRAD_BF16;
        if (t.m_scale != nullptr) {
            if (bf)
                adam_block_any<true, true>(t, b0, lane, sc);
            else
                adam_block_any<true, false>(t, b0, lane, sc);
        } else if (bf) {
            adam_block_any<false, true>(t, b0, lane, sc);
        } else {
            adam_block_any<false, false>(t, b0, lane, sc);
        }
    }
}

// Tensors [t0, t0 + count) as one launch.
template <int CAP>
cudaError_t adam_launch(const AdamTensor* ts, int count, AdamArgs a, bool update, int* ctas, cudaStream_t s, bool pdl) {
    AdamList<CAP> l;
    long long chunks = 0;
    for (int i = 0; i < count; ++i) {
        l.t[i] = ts[i];
        l.first[i] = (int)chunks;
        chunks += (ts[i].n + kAdamChunk - 1) / kAdamChunk;
    }
    l.first[count] = (int)chunks;
    l.count = count;
    if (!update) {
        // (without clipping only the CTA that advances the step)
        const long long most = (long long)kAdamNormCtas * block_gemm_sms();
        a.norm_group = (int)std::max(1LL, std::min(8LL, chunks / most));
        *ctas = a.max_norm > 0.f ? (int)std::min((chunks + a.norm_group - 1) / a.norm_group, most) : 0;
        return launch_ex(adamw_norm_kernel<CAP>, dim3((unsigned)(*ctas + (a.advance ? 1 : 0))), dim3(kAdamThreads), 0, s, pdl, l, a);
    }
    // 64 CTAs an SM, 16 times what is resident: handed out in order as others
    // end, they keep to one region of memory (562M values: 2.45 ms, 2.63 with as
    // many as are resident; from 512 on each one's first look at the norm shows)
    const long long grid = std::max(1LL, std::min<long long>(chunks, 64LL * block_gemm_sms()));
    return launch_ex(adamw_update_kernel<CAP>, dim3((unsigned)grid), dim3(kAdamThreads), 0, s, pdl, l, a);
}

cudaError_t adam_launch_any(const AdamTensor* ts, int count, const AdamArgs& a, bool update, int* ctas, cudaStream_t s,
                            bool pdl) {
    return count <= kAdamCapSmall ? adam_launch<kAdamCapSmall>(ts, count, a, update, ctas, s, pdl)
                                  : adam_launch<kAdamCap>(ts, count, a, update, ctas, s, pdl);
}

}  // namespace

long long adam_chunks(long long n) { return (n + kAdamChunk - 1) / kAdamChunk; }

size_t adam_scratch_bytes(int count) {
    const size_t launches = (size_t)(count + kAdamCap - 1) / kAdamCap;
    return 256 + (launches * kAdamNormCtas * kBlockSmsBound * sizeof(float4) + 255) / 256 * 256;
}

cudaError_t launch_adamw_norm(const AdamTensor* ts, int count, const AdamArgs& a, int* ctas, cudaStream_t s, bool pdl) {
    return adam_launch_any(ts, count, a, false, ctas, s, pdl);
}
cudaError_t launch_adamw_update(const AdamTensor* ts, int count, const AdamArgs& a, cudaStream_t s, bool pdl) {
    int ctas = 0;
    return adam_launch_any(ts, count, a, true, &ctas, s, pdl);
}

}  // namespace lrs

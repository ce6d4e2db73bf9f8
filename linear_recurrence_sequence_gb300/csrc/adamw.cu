// AdamW over many tensors at once, with the gradient norm and its clipping.
//
//   N = sqrt(sum g^2) over every tensor; k = min(1, max_norm / N)
//   m = b1 m + (1 - b1) k g;  v = b2 v + (1 - b2) (k g)^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Two launches: the norm (every gradient once; without clipping one CTA that
// only advances the step) and the update.  The list of tensors travels in the
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
// Bound by bandwidth: 30 bytes a value with 32-bit states, a BF16 parameter
// and its FP32 master, 18 with 8-bit states.  A warp takes 256 consecutive
// values (an 8-bit block), a lane four and four, so that every array is read
// and written in whole 128-byte lines.
#include <algorithm>

#include <cuda_fp8.h>

#include "kernels.cuh"

namespace lrs {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                             // values a scale stands for, values of a warp
constexpr int kAdamChunk = kAdamBlock * kAdamThreads / 32;  // values of a CTA at a time
constexpr float kFp8Max = 448.f;
constexpr float kFp8Tiny = 0.001953125f;                    // 2^-9, the smallest E4M3 value above 0
constexpr float kAdamSmall = 7.888609052210118e-31f;        // 2^-100

// The list of one launch, in the kernel's parameters.
template <int CAP>
struct AdamList {
    AdamTensor t[CAP];
    int first[CAP + 1];   // first chunk of each tensor; [count]: the chunks in all
    int count;
};

// The tensor of chunk c, searched on from tensor i (chunks come in ascending order).
template <int CAP>
__device__ __forceinline__ int adam_find(const AdamList<CAP>& l, int c, int i) {
    while (c >= l.first[i + 1]) ++i;
    return i;
}

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
// Four values from i on of an array of n (zeros past its end).
__device__ __forceinline__ void load_f32(const float* p, long long i, long long n, float (&v)[4]) {
    if (i + 4 <= n) {
        load4(p + i, v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < n ? p[i + k] : 0.f;
    }
}
__device__ __forceinline__ void store_f32(float* p, long long i, long long n, const float (&v)[4]) {
    if (i + 4 <= n) {
        *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[i + k] = v[k];
    }
}
__device__ __forceinline__ void load_bf16(const uint16_t* p, long long i, long long n, float (&v)[4]) {
    if (i + 4 <= n) {
        const uint2 q = *reinterpret_cast<const uint2*>(p + i);
        const float2 a = bf2_to_f2(q.x), b = bf2_to_f2(q.y);
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < n ? __uint_as_float((uint32_t)p[i + k] << 16) : 0.f;
    }
}
__device__ __forceinline__ void store_bf16(uint16_t* p, long long i, long long n, const float (&v)[4]) {
    const uint2 q = make_uint2(f2_to_bf2(v[0], v[1]), f2_to_bf2(v[2], v[3]));
    if (i + 4 <= n) {
        *reinterpret_cast<uint2*>(p + i) = q;
    } else {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[i + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
    }
}
__device__ __forceinline__ void load_fp8(const uint8_t* p, long long i, long long n, float s, float (&v)[4]) {
    uint32_t q = 0;
    if (i + 4 <= n) {
        q = *reinterpret_cast<const uint32_t*>(p + i);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) q |= (uint32_t)p[i + k] << (8 * k);
    }
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> (8 * k)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[k] = f.x * s;
        v[k + 1] = f.y * s;
    }
}
__device__ __forceinline__ void store_fp8(uint8_t* p, long long i, long long n, const float (&v)[4]) {
    const uint32_t q = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3) |
                       (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3) << 16;
    if (i + 4 <= n) {
        *reinterpret_cast<uint32_t*>(p + i) = q;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[i + k] = (uint8_t)(q >> (8 * k));
    }
}

// Sum over the CTA in a fixed order; the result in every thread.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kAdamThreads / 32; ++w) v += red[w];
    return v;
}

// b^t for t >= 1 by repeated squaring.
__device__ double adam_pow(double b, int t) {
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

// First launch of a step: sums of squares of the gradients (one partial sum a
// CTA), and in the first CTA the step's count and bias corrections.
template <int CAP>
__global__ void __launch_bounds__(kAdamThreads) adamw_norm_kernel(const __grid_constant__ AdamList<CAP> l,
                                                                  const AdamArgs a) {
    __shared__ float red[kAdamThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    pdl_wait();
    if (a.advance && blockIdx.x == 0 && threadIdx.x == 0) {
        const int t = *a.step + 1;
        *a.step = t;
        a.bias[0] = (float)(1.0 / (1.0 - adam_pow(a.beta1, t)));
        a.bias[1] = (float)(1.0 / (1.0 - adam_pow(a.beta2, t)));
    }
    if (a.max_norm <= 0.f) return;
    float s = 0.f;
    int i = 0;
    for (int c = (int)blockIdx.x; c < l.first[l.count]; c += (int)gridDim.x) {
        i = adam_find(l, c, i);
        const AdamTensor& t = l.t[i];
        const long long at = (long long)(c - l.first[i]) * kAdamChunk + warp * kAdamBlock + 4 * lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long e = at + 128 * k;
            if (e >= t.n) continue;
            float g[4];
            if (t.grad_dtype == LRS_GRAD_BF16)
                load_bf16(static_cast<const uint16_t*>(t.grad), e, t.n, g);
            else
                load_f32(static_cast<const float*>(t.grad), e, t.n, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = fmaf(g[j], g[j], s);
        }
    }
    s = cta_sum(s, red);
    if (threadIdx.x == 0) a.partial[a.partial0 + blockIdx.x] = s;
}

template <int CAP>
__global__ void __launch_bounds__(kAdamThreads) adamw_update_kernel(const __grid_constant__ AdamList<CAP> l,
                                                                    const AdamArgs a) {
    __shared__ float red[kAdamThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    pdl_wait();
    float clip = 1.f;
    if (a.max_norm > 0.f) {
        float s = 0.f;
        for (int i = threadIdx.x; i < a.partials; i += kAdamThreads) s += __ldcg(a.partial + i);
        const float norm = sqrtf(cta_sum(s, red));
        const bool skip = !(norm <= 3.4028234e38f);
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.advance) {
            *a.norm = norm;
            if (skip) *a.step -= 1;   // no other CTA of a skipped step reads it
        }
        if (skip) return;
        clip = norm > a.max_norm ? a.max_norm / norm : 1.f;
    }
    const float lr = __ldg(a.lr), ibc1 = __ldcg(a.bias), ibc2 = __ldcg(a.bias + 1);
    const float b1 = (float)a.beta1, c1 = (float)(1.0 - a.beta1), b2 = (float)a.beta2, c2 = (float)(1.0 - a.beta2);
    int i = 0;
    for (int c = (int)blockIdx.x; c < l.first[l.count]; c += (int)gridDim.x) {
        i = adam_find(l, c, i);
        const AdamTensor& t = l.t[i];
        const long long n = t.n;
        const long long b0 = (long long)(c - l.first[i]) * kAdamChunk + warp * kAdamBlock;
        if (b0 >= n) continue;
        const bool q8 = t.m_scale != nullptr;
        float* p32 = t.master != nullptr ? t.master : static_cast<float*>(t.param);
        float p[2][4], g[2][4], m[2][4], v[2][4];
        float ms = 0.f, vs = 0.f;
        if (q8) {
            ms = t.m_scale[b0 / kAdamBlock];
            vs = t.v_scale[b0 / kAdamBlock];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long e = b0 + 128 * k + 4 * lane;
            if (t.grad_dtype == LRS_GRAD_BF16)
                load_bf16(static_cast<const uint16_t*>(t.grad), e, n, g[k]);
            else
                load_f32(static_cast<const float*>(t.grad), e, n, g[k]);
            load_f32(p32, e, n, p[k]);
            if (q8) {
                load_fp8(static_cast<const uint8_t*>(t.m), e, n, ms, m[k]);
                load_fp8(static_cast<const uint8_t*>(t.v), e, n, vs, v[k]);
            } else {
                load_f32(static_cast<const float*>(t.m), e, n, m[k]);
                load_f32(static_cast<const float*>(t.v), e, n, v[k]);
            }
        }
        const float keep = 1.f - lr * t.weight_decay;
        float mt = 0.f, vt = 0.f, root[2][4];
        uint32_t mtop = 0u, vtop = 0u;   // magnitudes as integers: their order is the values', NaN above all
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float gg = g[k][j] * clip;
                const float vv = q8 ? v[k][j] * v[k][j] : v[k][j];
                // each product rounded by itself, as written above
                m[k][j] = __fadd_rn(__fmul_rn(m[k][j], b1), __fmul_rn(gg, c1));
                v[k][j] = __fadd_rn(__fmul_rn(vv, b2), __fmul_rn(__fmul_rn(gg, gg), c2));
                const float step = m[k][j] * ibc1 / (sqrtf(v[k][j] * ibc2) + a.eps);
                p[k][j] = fmaf(-lr, step, p[k][j] * keep);
                if (q8) {
                    root[k][j] = sqrtf(v[k][j]);
                    mtop = max(mtop, __float_as_uint(fabsf(m[k][j])));
                    vtop = max(vtop, __float_as_uint(root[k][j]));
                }
            }
        }
        if (q8) {
            mt = __uint_as_float(__reduce_max_sync(0xffffffffu, mtop));
            vt = __uint_as_float(__reduce_max_sync(0xffffffffu, vtop));
            const float mi = mt >= kAdamSmall ? kFp8Max / mt : 0.f, vi = vt >= kAdamSmall ? kFp8Max / vt : 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    m[k][j] *= mi;
                    const float r = root[k][j] * vi;
                    v[k][j] = r > 0.f ? fmaxf(r, kFp8Tiny) : r;
                }
            if (lane == 0) {
                t.m_scale[b0 / kAdamBlock] = mt >= kAdamSmall ? mt / kFp8Max : 0.f;
                t.v_scale[b0 / kAdamBlock] = vt >= kAdamSmall ? vt / kFp8Max : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long e = b0 + 128 * k + 4 * lane;
            if (e >= n) continue;
            store_f32(p32, e, n, p[k]);
            if (t.master != nullptr) store_bf16(static_cast<uint16_t*>(t.param), e, n, p[k]);
            if (q8) {
                store_fp8(static_cast<uint8_t*>(t.m), e, n, m[k]);
                store_fp8(static_cast<uint8_t*>(t.v), e, n, v[k]);
            } else {
                store_f32(static_cast<float*>(t.m), e, n, m[k]);
                store_f32(static_cast<float*>(t.v), e, n, v[k]);
            }
        }
    }
}

int adam_norm_ctas(long long chunks) {
    return (int)std::max(1LL, std::min<long long>(chunks, 4LL * block_gemm_sms()));
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
        *ctas = a.max_norm > 0.f ? adam_norm_ctas(chunks) : 1;
        return launch_ex(adamw_norm_kernel<CAP>, dim3((unsigned)*ctas), dim3(kAdamThreads), 0, s, pdl, l, a);
    }
    const long long grid = std::max(1LL, std::min<long long>(chunks, 4LL * block_gemm_sms()));
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
    return 256 + (launches * 4 * kBlockSmsBound * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_adamw_norm(const AdamTensor* ts, int count, const AdamArgs& a, int* ctas, cudaStream_t s, bool pdl) {
    return adam_launch_any(ts, count, a, false, ctas, s, pdl);
}
cudaError_t launch_adamw_update(const AdamTensor* ts, int count, const AdamArgs& a, cudaStream_t s, bool pdl) {
    int ctas = 0;
    return adam_launch_any(ts, count, a, true, &ctas, s, pdl);
}

}  // namespace lrs

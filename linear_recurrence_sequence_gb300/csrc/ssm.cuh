// What the forward, backward and step kernels of the selective state space
// scan share: the tile of channels and states of a warp, the time tile in
// shared memory, the step softplus(raw).
#pragma once

#include <atomic>
#include <cfloat>

#include "kernels.cuh"

namespace lrs {

// A warp owns 128 / LN channels: LN lanes share four channels, 8 states each,
// so a lane holds 4 x 8 states of one chunk of time in registers, as pairs of
// channels (FP32 arithmetic is two wide).  LN = 1, 2, 4, 8 for up to 8, 16, 32,
// 64 states a channel.  32 states a lane are what makes the operands cheap: a
// token's steps and inputs are 8 words of shared memory a lane, its b and c 8
// each, which lie there twice, as the pairs that the arithmetic takes; and the
// sum over the states of a channel crosses LN lanes only.
constexpr int kSsmCh = 4;        // channels of a lane
constexpr int kSsmSt = 8;        // states of a lane
constexpr int kSsmVec = kSsmSt;   // its states as float4, four channels each

template <int LN>
struct SsmWarp {
    static constexpr int CW = 32 / LN * kSsmCh;   // channels of a warp
    static constexpr int NP = kSsmSt * LN;        // states of a channel, padded
    static constexpr int RL = CW / 8;             // lanes that span a row of channels, 16 bytes each
    static constexpr int RPI = 32 / RL;           // rows that a warp's load instruction takes
};

// Lets `fn` use `most` bytes of dynamic shared memory, once per device (every
// launch of a kernel names the same bytes, whatever it uses of them).
inline cudaError_t allow_smem(const void* fn, size_t most, std::atomic<bool>* allowed) {
    int dev = 0;
    const cudaError_t de = cudaGetDevice(&dev);
    if (de != cudaSuccess) return de;
    const bool known = dev >= 0 && dev < 64;
    if (known && allowed[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess && known) allowed[dev].store(true, std::memory_order_release);
    return e;
}

// softplus(r) = max(r, 0) + log1p(e^-|r|): relative error within 2^-21 + 2^-23 max(-r, 0)
// (the second from the rounding of the exponential's argument), also where
// it is far below 1 (the logarithm of 1 + w would lose w's digits).
__device__ __forceinline__ f2x softplus2(f2x raw) {
    // log1p(w) / w on [0, 1] within 2.4e-8 of itself (a polynomial of degree 9)
    constexpr float kLog1p[10] = {1.000000000e+00f,  -4.999990165e-01f, 3.332996368e-01f, -2.495413423e-01f,
                                  1.967593879e-01f,  -1.530559212e-01f, 1.060365364e-01f, -5.695952475e-02f,
                                  1.985145733e-02f,  -3.244024236e-03f};
    float a, b;
    up2(raw, a, b);
    const f2x w = pk2(ex2_approx(-fabsf(a) * kLog2e), ex2_approx(-fabsf(b) * kLog2e));
    f2x p = dup2(kLog1p[9]);
#pragma unroll
    for (int i = 8; i >= 0; --i) p = fma2(p, w, dup2(kLog1p[i]));
    return fma2(p, w, pk2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}

// 1 / (1 + e^-r) within 2^-20 + 2^-23 max(-r, 0); 0 where it is below 2^-126.
__device__ __forceinline__ float ssm_sigmoid(float r) { return rcp_approx(1.f + ex2_approx(-r * kLog2e)); }

// A rate (negative), FP32's largest in place of infinity, whose product with a step of 0 would be NaN.  NaN stays.
__device__ __forceinline__ float finite_rate(float r) {
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(r), "f"(-FLT_MAX));
    return o;
}
// log2 of what a state keeps in a unit of time: -e^a_log log2 e.
__device__ __forceinline__ float ssm_rate(float a_log) { return finite_rate(-expf(a_log) * kLog2e); }

// 8 BF16 values as FP32 pairs.
__device__ __forceinline__ void unpack_pairs(const uint4 q, f2x (&v)[4]) {
    v[0] = bf2x(q.x);
    v[1] = bf2x(q.y);
    v[2] = bf2x(q.z);
    v[3] = bf2x(q.w);
}
// 8 floats of a vector, or zeros.
__device__ __forceinline__ void load_pairs(const float* p, bool on, f2x (&v)[4]) {
    if (p == nullptr || !on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = 0ull;
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = pk2(a.x, a.y);
    v[1] = pk2(a.z, a.w);
    v[2] = pk2(b.x, b.y);
    v[3] = pk2(b.z, b.w);
}
__device__ __forceinline__ void store_pairs(float* p, const f2x (&v)[4]) {
    float4 a, b;
    up2(v[0], a.x, a.y);
    up2(v[1], a.z, a.w);
    up2(v[2], b.x, b.y);
    up2(v[3], b.z, b.w);
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
}
// The same to global memory: 32 bytes at once where they may be (two 16-byte stores of a warp would each fill half of
// every sector that they touch).
__device__ __forceinline__ void put_pairs(float* p, const f2x (&v)[4]) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) != 0) {
        store_pairs(p, v);
        return;
    }
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]) : "memory");
}
__device__ __forceinline__ void read_pairs(const float* p, f2x (&v)[4]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = pk2(a.x, a.y);
    v[1] = pk2(a.z, a.w);
    v[2] = pk2(b.x, b.y);
    v[3] = pk2(b.z, b.w);
}
// A lane's states: [state][pair of channels].
typedef f2x SsmStates[kSsmSt][kSsmCh / 2];
__device__ __forceinline__ void clear_states(SsmStates& h) {
#pragma unroll
    for (int j = 0; j < kSsmSt; ++j) h[j][0] = h[j][1] = 0ull;
}
// Two of a token's b or c, each as a pair of equal values.
__device__ __forceinline__ void read_twice(const float* p, f2x& v0, f2x& v1) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v0 = pk2(q.x, q.y);
    v1 = pk2(q.z, q.w);
}
// A lane's four channels as pairs.
__device__ __forceinline__ void read_channels(const float* p, f2x (&v)[2]) { read_twice(p, v[0], v[1]); }

__device__ __forceinline__ float bf_up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Copies into shared memory that run on while the warp computes; `bytes` 0 writes zeros.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Asks for nt rows (of T) of the warp's channels, zeros past nt and D.  p: the
// first row's place of the warp's first channel.
template <int LN, int T>
__device__ __forceinline__ void ask_rows(const uint16_t* p, long long st, int nt, int width, uint16_t* dst, int lane) {
    using W = SsmWarp<LN>;
    constexpr int IT = (T + W::RPI - 1) / W::RPI;
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL, off = r0 * (int)st + c8;
    uint16_t* d = dst + r0 * W::CW + c8;
    if (nt == T && width >= W::CW) {
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (T % W::RPI == 0 || r0 < T) copy16(d + i * W::RPI * W::CW, p + i * W::RPI * (int)st + off, true);
        return;
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const bool on = c8 < width && r0 + i * W::RPI < nt;
        if (T % W::RPI == 0 || r0 < T) copy16(d + i * W::RPI * W::CW, on ? p + i * W::RPI * (int)st + off : p, on);
    }
}
// nt rows of b or c, two states at a time (SsmArgs.words).
template <int LN, int T>
__device__ __forceinline__ void ask_states(const uint16_t* p, long long st, int nt, int N, uint16_t* dst, int lane) {
    constexpr int NP = SsmWarp<LN>::NP;
#pragma unroll
    for (int k = 0; k < (T * NP / 2 + 31) / 32; ++k) {
        const int i = k * 32 + lane, t = i / (NP / 2), n = i % (NP / 2) * 2;
        const bool on = t < nt && n < N;
        if (T * NP / 2 % 32 == 0 || t < T) copy4(dst + 2 * i, on ? p + t * (int)st + n : p, on);
    }
}
// Where two of a token's b or c wait (states j and j + 1 of lane ln, every value twice): the LN lanes' side by side, so that
// they read them without a bank conflict (64 states, 4 x 4096 x 256: a lane's states in a row 236 us
// forward and 718 with the backward, so 169 and 533).
template <int LN>
__device__ __forceinline__ constexpr int state_at(int ln, int j) {
    return 4 * (j / 2 * LN + ln);
}
// The rows as FP32, in that order: from what ask_states brought, or (not `words`) a value at a time.
template <int LN, int T>
__device__ __forceinline__ void stage_states(const uint16_t* p, long long st, bool words, int nt, int N, const uint16_t* raw,
                                             float* dst, int lane) {
    constexpr int NP = SsmWarp<LN>::NP, K = (T * NP / 2 + 31) / 32;
    uint32_t v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = k * 32 + lane, t = i / (NP / 2), q = i % (NP / 2), n = q % LN * kSsmSt + q / LN * 2;
        v[k] = 0u;
        if (T * NP / 2 % 32 != 0 && t >= T) continue;
        if (words) {
            v[k] = *reinterpret_cast<const uint32_t*>(raw + t * NP + n);
        } else {
            uint32_t lo = 0u, hi = 0u;
            if (t < nt && n < N) lo = __ldg(p + t * (int)st + n);
            if (t < nt && n + 1 < N) hi = __ldg(p + t * (int)st + n + 1);
            v[k] = lo | hi << 16;
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (T * NP / 2 % 32 == 0 || k * 32 + lane < T * NP / 2) {
            const float2 f = bf2_to_f2(v[k]);
            reinterpret_cast<float4*>(dst)[k * 32 + lane] = make_float4(f.x, f.x, f.y, f.y);
        }
}
// delta_bias of the warp's channels.
template <int LN>
__device__ __forceinline__ void stage_bias(const float* bias, int c0, int D, float* dst, int lane) {
#pragma unroll
    for (int i = lane; i < SsmWarp<LN>::CW; i += 32) dst[i] = bias != nullptr && c0 + i < D ? __ldg(bias + c0 + i) : 0.f;
}

// The warp's number in its CTA, the same in all its lanes for the compiler too.
__device__ __forceinline__ int warp_of() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

struct SsmPlace {
    int b, chunk, group, warp;
    bool on;
};
// CTAs: chunk by chunk (`chunks` of a row, from number `first` on), then the groups of a row side by side (they share b
// and c in L1).
__device__ __forceinline__ SsmPlace place(const SsmArgs& a, int chunks, int first) {
    SsmPlace p;
    const long long i = blockIdx.x;
    const int gq = (int)(i % a.ngq);
    const long long r = i / a.ngq;
    p.chunk = first + (int)(r % chunks);
    p.b = (int)(r / chunks);
    p.warp = warp_of();
    p.group = gq * (blockDim.x >> 5) + p.warp;
    p.on = p.group < a.groups;
    return p;
}

// The first of the rows of batch row b from token t on, from channel c on.
__device__ __forceinline__ const uint16_t* row_at(const SsmRows& r, int b, int t, int c) {
    return r.p + (long long)b * r.sb + (long long)t * r.st + c;
}

// A lane's 4 x 8 values of a [D][N] matrix, zeros past D and N.  quads: N is a multiple of 4 and the matrix on a 16-byte
// boundary (a lane's 8 values of a channel are one sector; one at a time they cost 8 times the L1 traffic).
__device__ __forceinline__ void load_states(const float* m, bool quads, int c0, int n0, int D, int N, float (&v)[kSsmCh][kSsmSt]) {
    const float* p = m + (long long)c0 * N + n0;
#pragma unroll
    for (int i = 0; i < kSsmCh; ++i) {
        if (quads) {
#pragma unroll
            for (int j = 0; j < kSsmSt; j += 4) {
                float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + i < D && n0 + j < N) q = __ldg(reinterpret_cast<const float4*>(p + i * N + j));
                v[i][j] = q.x;
                v[i][j + 1] = q.y;
                v[i][j + 2] = q.z;
                v[i][j + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSsmSt; ++j) v[i][j] = c0 + i < D && n0 + j < N ? __ldg(p + i * N + j) : 0.f;
        }
    }
}
// The rates of a lane's states (1 past N and D, where the states and all that is added to them are zeros; ZERO: 0 there).
template <bool ZERO = false>
__device__ __forceinline__ void load_rates(const float* a_log, bool quads, int c0, int n0, int D, int N, SsmStates& A) {
    float v[kSsmCh][kSsmSt];
    load_states(a_log, quads, c0, n0, D, N, v);
#pragma unroll
    for (int i = 0; i < kSsmCh; ++i)
#pragma unroll
        for (int j = 0; j < kSsmSt; ++j) v[i][j] = !ZERO || (c0 + i < D && n0 + j < N) ? ssm_rate(v[i][j]) : 0.f;
#pragma unroll
    for (int j = 0; j < kSsmSt; ++j) {
        A[j][0] = pk2(v[0][j], v[1][j]);
        A[j][1] = pk2(v[2][j], v[3][j]);
    }
}

// A lane's states from and to [.., D, N] rows of FP32.
__device__ __forceinline__ void load_state(const float* s, bool quads, long long row, int c0, int n0, int D, int N, SsmStates& h) {
    clear_states(h);
    if (s == nullptr) return;
    float v[kSsmCh][kSsmSt];
    load_states(s + row * D * N, quads, c0, n0, D, N, v);
#pragma unroll
    for (int j = 0; j < kSsmSt; ++j) {
        h[j][0] = pk2(v[0][j], v[1][j]);
        h[j][1] = pk2(v[2][j], v[3][j]);
    }
}
__device__ __forceinline__ void store_state(float* s, bool quads, long long row, int c0, int n0, int D, int N, const SsmStates& h) {
    float v[kSsmCh][kSsmSt];
#pragma unroll
    for (int j = 0; j < kSsmSt; ++j) {
        up2(h[j][0], v[0][j], v[1][j]);
        up2(h[j][1], v[2][j], v[3][j]);
    }
    float* p = s + (row * D + c0) * N + n0;
#pragma unroll
    for (int i = 0; i < kSsmCh; ++i) {
        if (quads) {
#pragma unroll
            for (int j = 0; j < kSsmSt; j += 4)
                if (c0 + i < D && n0 + j < N)
                    *reinterpret_cast<float4*>(p + i * N + j) = make_float4(v[i][j], v[i][j + 1], v[i][j + 2], v[i][j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < kSsmSt; ++j)
                if (c0 + i < D && n0 + j < N) p[i * N + j] = v[i][j];
        }
    }
}
// The same in the kernels' own layout: [kSsmVec][32 lanes] float4 for a warp.
__device__ __forceinline__ void load_tile_state(const float4* p, int lane, SsmStates& h) {
#pragma unroll
    for (int k = 0; k < kSsmVec; ++k) {
        const float4 v = __ldcg(p + k * 32 + lane);
        h[k][0] = pk2(v.x, v.y);
        h[k][1] = pk2(v.z, v.w);
    }
}
__device__ __forceinline__ void store_tile_state(float4* p, int lane, const SsmStates& h) {
#pragma unroll
    for (int k = 0; k < kSsmVec; ++k) {
        float4 v;
        up2(h[k][0], v.x, v.y);
        up2(h[k][1], v.z, v.w);
        p[k * 32 + lane] = v;
    }
}

// The GPU's exponential is 1.7e-8 to 2.6e-8 too small on average between 2^-0.06 and 2^-0.003 (5e-9 from there to 1), a
// loss that a state adds up over all the tokens that it keeps.  So much more in the exponent takes half of it away, in the
// same instruction, and leaves 2^0 = 1 (1 x 32768 x 2048, 16 states: da_log 1.45e-6 off the definition, so 8.0e-7).
constexpr float kEx2Low = 2e-8f;
// a = e^(A dt)
__device__ __forceinline__ f2x decay(f2x A, f2x dt) {
    float e0, e1;
    up2(fma2(A, dt, dup2(kEx2Low)), e0, e1);
    return pk2(ex2_approx(e0), ex2_approx(e1));
}

// The sum of v[c] over the LN lanes that share a channel; lane ln of them ends
// with the sums of the channels [ln 4 / LN, ...) in v[0 ..] (LN = 8: lanes 2 c and 2 c + 1 with channel c's).
template <int LN>
__device__ __forceinline__ void sum_states(const f2x (&v2)[2], float (&v)[kSsmCh], int lane) {
    up2(v2[0], v[0], v[1]);
    up2(v2[1], v[2], v[3]);
    if (LN == 1) return;
    int keep = kSsmCh;
#pragma unroll
    for (int m = LN / 2; m >= 1; m >>= 1) {
        if (keep > 1) {
            keep >>= 1;
            const bool up = lane & m;
#pragma unroll
            for (int i = 0; i < keep; ++i) {
                const float send = up ? v[i] : v[i + keep], mine = up ? v[i + keep] : v[i];
                v[i] = mine + __shfl_xor_sync(0xffffffffu, send, m);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
}
// Writes what sum_states left to the warp's row of channels.
template <int LN>
__device__ __forceinline__ void put_channels(float* row, const float (&v)[kSsmCh], int lc, int ln) {
    float* p = row + lc * kSsmCh;
    if (LN == 1) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    if (LN == 2) *reinterpret_cast<float2*>(p + 2 * ln) = make_float2(v[0], v[1]);
    if (LN == 4) p[ln] = v[0];
    if (LN == 8) p[ln >> 1] = v[0];
}

// Bit t: a sequence starts at token t0 + t (t < nt <= 32).
__device__ __forceinline__ uint32_t start_bits(const uint8_t* reset, long long row, int nt, int lane) {
    if (reset == nullptr) return 0u;
    return __ballot_sync(0xffffffffu, lane < nt && __ldg(reset + row + lane) != 0);
}

}  // namespace lrs

// The norms before and after a residual branch, fused with its gate and its
// scale: the join of a bare mixer (its output y, its gate branch g) with the
// residual stream x, and the norm that feeds the next layer.
//
//   p = y rstd1, n = p gamma_post, u = scale GeLU(g) n, r = x + u
//   q = r rstd2, h = q gamma_pre      rstd = 1 / sqrt(mean^2 + eps) of y, of r
//
// Backward for dr, dh (means over the row):
//   a = dh gamma_pre, dx = dr + rstd2 (a - q mean(a q))
//   e = dx GeLU(g);  dg = dx scale gamma_post p GeLU'(g)
//   b = e scale gamma_post, dy = rstd1 (b - p mean(b p))
//   dgamma_pre = sum dh q, A = sum e p, dscale = gamma_post A, dgamma_post = scale A
// (a channel's scale and gamma_post leave the sum over the rows, so the two
// gradients share one sum).
// r is formed again from x, y and g, in FP32: the rounded r is not read.
//
// Bound by bandwidth: 10 bytes a value forward, 16 backward, each array once
// (16384 x 1024 with branch and gate, events around each launch: 30 us, 5.6 TB/s,
// and 48 us, 5.5 TB/s; 5001 x 2560 without a branch 12 and 22 us; 16 rows of 2048
// in a graph 2.4 us).
// A thread holds 8 consecutive channels (16 bytes of each operand) of a row
// that stays in registers between its two row sums; a CTA takes several rows
// at a time where they are narrow.  Where a CTA has more than one group of
// rows to go through, the groups arrive by bulk copies in a ring of shared
// memory, so that the loads run ahead of the row sums' barriers; a call with
// few rows loads them directly (no barriers to set up: a decoding step).
// The two sums add up in registers over the rows of a thread, then over the
// CTA's row slots in shared memory, one partial row a CTA, joined in a fixed
// order by a second kernel.
#include <algorithm>
#include <atomic>

#include "kernels.cuh"

namespace lrs {

namespace {

constexpr int kGnMaxThreads = 512;
constexpr int kGnMaxWarps = kGnMaxThreads / 32;
constexpr int kGnSmemMax = 216 * 1024;   // of the ring

// Pairs of channels in the two-wide FP32 instructions: the row arithmetic is
// half of what these kernels issue.
__device__ __forceinline__ uint64_t as_u64(float2 v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 as_f2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_f2(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ void unpack8(const uint4 q, float2 (&v)[4]) {
    v[0] = bf2_to_f2(q.x);
    v[1] = bf2_to_f2(q.y);
    v[2] = bf2_to_f2(q.z);
    v[3] = bf2_to_f2(q.w);
}
__device__ __forceinline__ uint4 pack8(const float2 (&v)[4]) {
    return make_uint4(f2_to_bf2(v[0].x, v[0].y), f2_to_bf2(v[1].x, v[1].y), f2_to_bf2(v[2].x, v[2].y),
                      f2_to_bf2(v[3].x, v[3].y));
}
// 8 channels of a vector; ones where it is missing or the thread has none.
__device__ __forceinline__ void load8(const float* p, int v, bool on, float2 (&o)[4]) {
    if (p == nullptr || !on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = both(1.f);
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(p) + 2 * v), b = __ldg(reinterpret_cast<const float4*>(p) + 2 * v + 1);
    o[0] = make_float2(a.x, a.y);
    o[1] = make_float2(a.z, a.w);
    o[2] = make_float2(b.x, b.y);
    o[3] = make_float2(b.z, b.w);
}
// scale gamma_post of 8 channels.
__device__ __forceinline__ void load_product(const float* p, const float* q, int v, bool on, float2 (&o)[4]) {
    float2 b[4];
    load8(p, v, on, o);
    load8(q, v, on, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul2(o[i], b[i]);
}

// The block's GeLU, x s with s = 1 / (1 + e^{-2u}), u = sqrt(2/pi) (x + 0.044715 x^3),
// from the SFU: e^{-2u} = 2^(x (k0 + k1 x^2)) and the reciprocal, 2^-20 relative
// over |2u| <= 20; six operations, where the block's own form takes about 15
// (the forward kernel was bound by them).  Its derivative is
// s (1 + (1 - s) x (k2 + k3 x^2)) with 1 - s = e^{-2u} s, formed at x held within
// kGeluEnd of 0: there e^{-2u} is 2^127.6 or its reciprocal, whose own reciprocals
// are exactly 0 (flushed) and 1, so that the derivative of any gate farther out is 0
// or 1 and no factor overflows.
constexpr float kGelu0 = -2.302208198f;    // -2 sqrt(2/pi) log2(e)
constexpr float kGelu1 = -0.1029432397f;   // 0.044715 of it
constexpr float kGelu2 = 1.595769122f;     // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.2140644488f;    // 3 0.044715 of it
constexpr float kGeluEnd = 10.05f;
// x, held within +-end (end > 0; NaN stays).
__device__ __forceinline__ float hold(float x, float end) {
    float r;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(end));
    return r;
}
__device__ __forceinline__ float2 gn_gelu(float2 x) {
    const float2 t = mul2(x, fma2(both(kGelu1), mul2(x, x), both(kGelu0)));
    const float2 e = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), both(1.f));
    return mul2(x, make_float2(rcp_approx(e.x), rcp_approx(e.y)));
}
__device__ __forceinline__ void gn_gelu_grad(float2 x, float2& g, float2& dg) {
    const float2 c = make_float2(hold(x.x, kGeluEnd), hold(x.y, kGeluEnd)), c2 = mul2(c, c);
    const float2 t = mul2(c, fma2(both(kGelu1), c2, both(kGelu0)));
    const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    const float2 e1 = add2(e, both(1.f));
    const float2 s = make_float2(rcp_approx(e1.x), rcp_approx(e1.y));
    g = mul2(x, s);
    dg = fma2(mul2(s, mul2(e, s)), mul2(c, fma2(both(kGelu3), c2, both(kGelu2))), s);
}

// Sum over the threads of a row (blockDim.x of them, whole warps).  `red` is
// this sum's own buffer, zeros past the row's warps: sums that follow each
// other use two buffers in turn, so one barrier each is enough.
__device__ __forceinline__ float row_sum(float v, float (*red)[kGnMaxWarps]) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.y][threadIdx.x >> 5] = v;
    __syncthreads();
    const float4* r = reinterpret_cast<const float4*>(red[threadIdx.y]);
    v = 0.f;
    for (int w = 0; w < (int)blockDim.x; w += 128, ++r) {
        const float4 q = *r;
        v += (q.x + q.y) + (q.z + q.w);
    }
    return v;
}

// A ring of row groups in shared memory: slot k of the ring holds NOPS
// operands of blockDim.y rows each, as they lie in memory.
template <int NOPS>
struct GnRing {
    const uint4* src[NOPS];
    long long T;
    int nv, stages, slot, asked;   // slot: of the current group; asked: of the next one to ask for
    uint32_t phase, op_bytes;
    long long next;                // first row of the next group to ask for
    uint8_t* buf;
    uint64_t* full;
    const uint8_t* mine;           // this thread's place in the current slot

    __device__ __forceinline__ void start(long long rows, int nv_, int stages_, uint8_t* buf_, uint64_t* full_) {
        T = rows;
        nv = nv_;
        stages = stages_;
        buf = buf_;
        full = full_;
        slot = asked = 0;
        phase = 0u;
        op_bytes = blockDim.y * (uint32_t)nv * 16u;
        next = (long long)blockIdx.x * blockDim.y;
        mine = buf + (threadIdx.y * (uint32_t)nv + threadIdx.x) * 16u;
        if (threadIdx.x == 0 && threadIdx.y == 0) {
            for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
            for (int i = 0; i < stages; ++i) ask();
        }
        __syncthreads();
    }
    // Thread 0: asks for the CTA's next group of rows (groups blockIdx.x, + gridDim.x, ...).
    __device__ __forceinline__ void ask() {
        if (next < T) {
            const uint32_t bytes = (uint32_t)min((long long)blockDim.y, T - next) * (uint32_t)nv * 16u;
            mbar_arrive_expect_tx(&full[asked], NOPS * bytes);
#pragma unroll
            for (int k = 0; k < NOPS; ++k)
                bulk_load(buf + (asked * NOPS + k) * op_bytes, src[k] + (size_t)next * nv, bytes, &full[asked]);
        }
        next += (long long)gridDim.x * blockDim.y;
        if (++asked == stages) asked = 0;
    }
    // Operand k of this thread's row, its group of channels `at` threads on.
    __device__ __forceinline__ uint4 get(int k, int at) const {
        return *reinterpret_cast<const uint4*>(mine + (slot * NOPS + k) * op_bytes + at * 16);
    }
    __device__ __forceinline__ bool wait() const { return mbar_wait_bounded(&full[slot], phase); }
    // Every thread has taken its operands (rows of one warp met no barrier in their sums): the slot is filled again.
    __device__ __forceinline__ void taken() {
        if (blockDim.x == 32) __syncthreads();
        if (threadIdx.x == 0 && threadIdx.y == 0) {
            fence_proxy_async();
            ask();
        }
        if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
        }
    }
};
// Zeroes the sums' buffers (the places past a row's warps stay zero).
__device__ __forceinline__ void clear_red(float (*red)[kGnMaxThreads / 32][kGnMaxWarps]) {
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 2 * (kGnMaxThreads / 32) * kGnMaxWarps;
         i += blockDim.x * blockDim.y)
        red[0][0][i] = 0.f;
    __syncthreads();
}
constexpr int kGnStagesMax = 4;

// VEC: groups of 8 channels per thread (group threadIdx.x + k blockDim.x).
// RING: the rows arrive in the ring; else one group of rows a CTA, loaded directly.
template <bool Y, bool G, int VEC, bool RING>
__global__ void __launch_bounds__(kGnMaxThreads) gated_norm_fwd_kernel(const GatedNormArgs a) {
    constexpr int NOPS = 1 + Y + G;
    __shared__ __align__(16) float red[2][kGnMaxThreads / 32][kGnMaxWarps];
    __shared__ __align__(8) uint64_t full[kGnStagesMax];
    extern __shared__ __align__(128) uint8_t buf[];
    pdl_trigger();
    pdl_wait();
    const int nv = a.D / 8;
    const float inv_d = 1.f / (float)a.D;
    if (blockDim.x > 32) clear_red(red);
    GnRing<NOPS> ring;
    if (RING) {
        ring.src[0] = a.x;
        if (Y) ring.src[Y] = a.y;
        if (G) ring.src[Y + G] = a.g;
        ring.start(a.T, nv, a.stages, buf, full);
    }
    // a thread's channels are the same in every row: so are its vectors
    float2 gm[VEC][4], sg[VEC][4];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        load8(a.gamma_pre, v, v < nv, gm[k]);
        if (Y) load_product(a.scale, a.gamma_post, v, v < nv, sg[k]);
    }
    bool lost = false;
    int it = 0;
    for (long long base = (long long)blockIdx.x * blockDim.y; base < a.T; base += (long long)gridDim.x * blockDim.y, ++it) {
        const long long row = base + threadIdx.y;
        uint4 qx[VEC], qy[VEC], qg[VEC];
        if (RING) lost |= !ring.wait();
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            const size_t o = (size_t)row * nv + v;
            qx[k] = qy[k] = qg[k] = make_uint4(0u, 0u, 0u, 0u);
            if (row < a.T && v < nv) {
                qx[k] = RING ? ring.get(0, k * blockDim.x) : __ldg(a.x + o);
                if (Y) qy[k] = RING ? ring.get(Y, k * blockDim.x) : __ldg(a.y + o);
                if (G) qg[k] = RING ? ring.get(Y + G, k * blockDim.x) : __ldg(a.g + o);
            }
        }
        float2 r[VEC][4];
        float rstd1 = 0.f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) unpack8(qx[k], r[k]);
        if (Y) {
            float2 ss = both(0.f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float2 y[4];
                unpack8(qy[k], y);
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fma2(y[i], y[i], ss);
            }
            rstd1 = rsqrtf(fmaf(row_sum(ss.x + ss.y, red[0]), inv_d, a.eps));
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float2 y[4], g[4];
                unpack8(qy[k], y);
                unpack8(qg[k], g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = mul2(mul2(y[i], both(rstd1)), sg[k][i]);
                    r[k][i] = G ? fma2(gn_gelu(g[i]), p, r[k][i]) : add2(r[k][i], p);
                }
            }
        }
        float2 ss = both(0.f);
#pragma unroll
        for (int k = 0; k < VEC; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = fma2(r[k][i], r[k][i], ss);
        float rstd2 = rsqrtf(fmaf(row_sum(ss.x + ss.y, red[Y ? 1 : it & 1]), inv_d, a.eps));
        if (lost) rstd1 = rstd2 = NAN;
        if (RING) ring.taken();
        if (row >= a.T) continue;
        if (threadIdx.x == 0 && a.rstd != nullptr)
            a.rstd[row] = make_float2(rstd1, rstd2);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v >= nv) continue;
            float2 h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = mul2(mul2(r[k][i], both(rstd2)), gm[k][i]);
            const size_t o = (size_t)row * nv + v;
            if (Y) a.r[o] = pack8(r[k]);
            a.h[o] = pack8(h);
        }
    }
}

template <bool Y, bool G, int VEC>
__global__ void __launch_bounds__(kGnMaxThreads) gated_norm_bwd_kernel(const GatedNormBwdArgs a) {
    constexpr int NOPS = 3 + Y + G;
    __shared__ __align__(16) float red[2][kGnMaxThreads / 32][kGnMaxWarps];
    __shared__ __align__(8) uint64_t full[kGnStagesMax];
    extern __shared__ __align__(128) uint8_t buf[];   // the ring, then the sums [2][rows][D]
    pdl_trigger();
    pdl_wait();
    const GatedNormArgs& f = a.f;
    const int nv = f.D / 8;
    const float inv_d = 1.f / (float)f.D;
    if (blockDim.x > 32) clear_red(red);
    GnRing<NOPS> ring;
    ring.src[0] = f.x;
    ring.src[1] = a.dh;
    ring.src[2] = a.dr != nullptr ? a.dr : a.dh;   // without dr its place is not read
    if (Y) ring.src[2 + Y] = f.y;
    if (G) ring.src[2 + Y + G] = f.g;
    ring.start(f.T, nv, f.stages, buf, full);
    // a thread's channels are the same in every row: so are its vectors
    float2 gm[VEC][4], sg[VEC][4];
    float2 dpre[VEC][4], sum[VEC][4];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        load8(f.gamma_pre, v, v < nv, gm[k]);
        if (Y) load_product(f.scale, f.gamma_post, v, v < nv, sg[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) dpre[k][i] = sum[k][i] = both(0.f);
    }
    // the rows' reciprocal norms, one group ahead
    float2 ahead = make_float2(0.f, 0.f);
    if ((long long)blockIdx.x * blockDim.y + threadIdx.y < f.T)
        ahead = __ldg(f.rstd + (long long)blockIdx.x * blockDim.y + threadIdx.y);
    bool lost = false;
    int it = 0;
    for (long long base = (long long)blockIdx.x * blockDim.y; base < f.T; base += (long long)gridDim.x * blockDim.y, ++it) {
        const long long row = base + threadIdx.y;
        uint4 qx[VEC], qy[VEC], qg[VEC], qr[VEC], qh[VEC];
        float2 rs = ahead;
        const long long after = row + (long long)gridDim.x * blockDim.y;
        ahead = after < f.T ? __ldg(f.rstd + after) : make_float2(0.f, 0.f);
        lost |= !ring.wait();
        if (lost) rs = make_float2(NAN, NAN);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            qx[k] = qy[k] = qg[k] = qr[k] = qh[k] = make_uint4(0u, 0u, 0u, 0u);
            if (row < f.T && v < nv) {
                qx[k] = ring.get(0, k * blockDim.x);
                qh[k] = ring.get(1, k * blockDim.x);
                if (a.dr != nullptr) qr[k] = ring.get(2, k * blockDim.x);
                if (Y) qy[k] = ring.get(2 + Y, k * blockDim.x);
                if (G) qg[k] = ring.get(2 + Y + G, k * blockDim.x);
            }
        }
        // q = r rstd2, a = dh gamma_pre, mean(a q)
        float2 q[VEC][4], ge[VEC][4], dge[VEC][4], s = both(0.f);
        const float2 rs1 = both(rs.x), rs2 = both(rs.y);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            float2 dh[4];
            unpack8(qx[k], q[k]);
            unpack8(qh[k], dh);
            if (Y) {
                float2 y[4], g[4];
                unpack8(qy[k], y);
                unpack8(qg[k], g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (G) {
                        gn_gelu_grad(g[i], ge[k][i], dge[k][i]);
                        q[k][i] = fma2(mul2(sg[k][i], ge[k][i]), mul2(y[i], rs1), q[k][i]);
                    } else {
                        q[k][i] = fma2(sg[k][i], mul2(y[i], rs1), q[k][i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[k][i] = mul2(q[k][i], rs2);
                const float2 dq = mul2(dh[i], q[k][i]);
                dpre[k][i] = add2(dpre[k][i], dq);
                s = fma2(dq, gm[k][i], s);
            }
        }
        const float mean = row_sum(s.x + s.y, red[Y ? 0 : it & 1]) * inv_d;
        ring.taken();
        float2 dx[VEC][4];
        s = both(0.f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            float2 dh[4], dr[4];
            unpack8(qh[k], dh);
            unpack8(qr[k], dr);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dx[k][i] = fma2(rs2, fma2(q[k][i], both(-mean), mul2(dh[i], gm[k][i])), dr[i]);
            if (row < f.T && v < nv) a.dx[(size_t)row * nv + v] = pack8(dx[k]);
            if (Y) {
                float2 y[4], dg[4];
                unpack8(qy[k], y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = mul2(y[i], rs1), e = G ? mul2(dx[k][i], ge[k][i]) : dx[k][i], ep = mul2(e, p);
                    if (G) dg[i] = mul2(mul2(dx[k][i], dge[k][i]), mul2(p, sg[k][i]));
                    sum[k][i] = add2(sum[k][i], ep);
                    s = fma2(ep, sg[k][i], s);
                    dx[k][i] = mul2(e, sg[k][i]);   // b
                }
                if (G && row < f.T && v < nv) a.dg[(size_t)row * nv + v] = pack8(dg);
            }
        }
        if (Y) {
            // dy = rstd1 b - y (rstd1^2 mean)
            const float mean1 = row_sum(s.x + s.y, red[1]) * inv_d;
            const float2 back = both(-rs.x * rs.x * mean1);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                float2 y[4], dy[4];
                unpack8(qy[k], y);
#pragma unroll
                for (int i = 0; i < 4; ++i) dy[i] = fma2(rs1, dx[k][i], mul2(y[i], back));
                if (row < f.T && v < nv) a.dy[(size_t)row * nv + v] = pack8(dy);
            }
        }
    }
    // the CTA's row slots in order, then one partial row of each sum (the ring
    // is drained: every group asked for has been waited for)
    __syncthreads();
    float* acc = reinterpret_cast<float*>(buf);
    const int sums = Y ? 2 : 1;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v >= nv) continue;
        float* o = acc + (size_t)threadIdx.y * f.D + 8 * v;
        const size_t stride = (size_t)blockDim.y * f.D;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            reinterpret_cast<float2*>(o)[i] = dpre[k][i];
            if (Y) reinterpret_cast<float2*>(o + stride)[i] = sum[k][i];
        }
    }
    __syncthreads();
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    for (int c = tid; c < sums * f.D; c += blockDim.x * blockDim.y) {
        const int w = c / f.D, d = c - w * f.D;
        float s = 0.f;
        for (int y = 0; y < (int)blockDim.y; ++y) s += acc[((size_t)w * blockDim.y + y) * f.D + d];
        a.part[((size_t)w * gridDim.x + blockIdx.x) * f.D + d] = s;
    }
}

// The partial rows of sum blockIdx.y joined: 32 columns a CTA, warp w the rows
// w, w + 32, ..., the warps' sums then in order.
__global__ void __launch_bounds__(1024) gated_norm_sum_kernel(const float* __restrict__ part, int parts, int D,
                                                              const float* __restrict__ gamma_post,
                                                              const float* __restrict__ scale, float* dgamma_pre,
                                                              float* dgamma_post, float* dscale) {
    __shared__ float acc[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* p = part + (size_t)blockIdx.y * parts * D;
    float s = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int i = w; i < parts; i += 32) s += __ldcg(p + (size_t)i * D + c);
    }
    acc[w][lane] = s;
    __syncthreads();
    if (w != 0 || c >= D) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += acc[i][lane];
    if (blockIdx.y == 0) {
        dgamma_pre[c] = s;
    } else {
        dscale[c] = s * (gamma_post != nullptr ? gamma_post[c] : 1.f);
        dgamma_post[c] = s * (scale != nullptr ? scale[c] : 1.f);
    }
}

struct GnShape {
    int vec;
    dim3 block;
};
// Whole warps of threads with 8 channels each span a row; narrow rows share a
// CTA of 256 threads.
GnShape gn_shape(int D) {
    GnShape s;
    const int nv = D / 8;
    s.vec = nv <= kGnMaxThreads ? 1 : 2;
    const int x = ((nv + s.vec - 1) / s.vec + 31) / 32 * 32;
    s.block = dim3((unsigned)x, (unsigned)std::max(1, 256 / x));
    return s;
}

// CTAs per SM that the registers leave room for, and the ring's stages: what
// fits beside them, two at least (a group of rows in flight while one is used).
int gn_ctas_per_sm(const GnShape& sh, int threads_per_sm) {
    return std::max(1, threads_per_sm / (int)(sh.block.x * sh.block.y));
}
int gn_stages(size_t group_bytes, int ctas_per_sm) {
    const size_t room = kGnSmemMax / ctas_per_sm;
    return (int)std::max<size_t>(2, std::min<size_t>(kGnStagesMax, room / group_bytes));
}

// Lets `fn` use `smem` bytes of dynamic shared memory; the largest size asked
// for so far is kept per device, so that a launch does not ask again.
cudaError_t gn_allow(const void* fn, int smem, std::atomic<int>* allowed) {
    int dev = 0;
    const cudaError_t de = cudaGetDevice(&dev);
    if (de != cudaSuccess) return de;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && allowed[dev].load(std::memory_order_acquire) >= smem) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kGnSmemMax);
    if (e == cudaSuccess && keep) allowed[dev].store(kGnSmemMax, std::memory_order_release);
    return e;
}

template <bool Y, bool G, int VEC>
cudaError_t gn_fwd_as(GatedNormArgs a, const GnShape& sh, cudaStream_t s, bool pdl) {
    const long long groups = (a.T + sh.block.y - 1) / sh.block.y;
    const int per_sm = gn_ctas_per_sm(sh, VEC == 2 ? 512 : Y ? 1024 : 1536);
    const long long resident = (long long)per_sm * block_gemm_sms();
    // one group of rows a CTA needs no ring
    if (groups <= resident)
        return launch_ex(gated_norm_fwd_kernel<Y, G, VEC, false>, dim3((unsigned)groups), sh.block, 0, s, pdl, a);
    const size_t group = (size_t)(1 + Y + G) * sh.block.y * a.D * 2;
    a.stages = gn_stages(group, per_sm);
    auto* fn = gated_norm_fwd_kernel<Y, G, VEC, true>;
    const size_t smem = group * a.stages;
    static std::atomic<int> allowed[64];
    const cudaError_t e = gn_allow(reinterpret_cast<const void*>(fn), (int)smem, allowed);
    if (e != cudaSuccess) return e;
    return launch_ex(fn, dim3((unsigned)resident), sh.block, smem, s, pdl, a);
}
template <bool Y, bool G>
cudaError_t gn_fwd(const GatedNormArgs& a, cudaStream_t s, bool pdl) {
    const GnShape sh = gn_shape(a.D);
    return sh.vec == 1 ? gn_fwd_as<Y, G, 1>(a, sh, s, pdl) : gn_fwd_as<Y, G, 2>(a, sh, s, pdl);
}

template <bool Y, bool G, int VEC>
cudaError_t gn_bwd_as(GatedNormBwdArgs a, const GnShape& sh, int ctas, cudaStream_t s, bool pdl) {
    const size_t group = (size_t)(3 + Y + G) * sh.block.y * a.f.D * 2;
    a.f.stages = gn_stages(group, gn_ctas_per_sm(sh, Y ? 512 : 1024));
    const size_t smem = std::max(group * a.f.stages, (size_t)(Y ? 2 : 1) * sh.block.y * a.f.D * sizeof(float));
    auto* fn = gated_norm_bwd_kernel<Y, G, VEC>;
    static std::atomic<int> allowed[64];
    const cudaError_t e = gn_allow(reinterpret_cast<const void*>(fn), (int)smem, allowed);
    if (e != cudaSuccess) return e;
    return launch_ex(fn, dim3((unsigned)ctas), sh.block, smem, s, pdl, a);
}
template <bool Y, bool G>
cudaError_t gn_bwd(const GatedNormBwdArgs& a, int ctas, cudaStream_t s, bool pdl) {
    const GnShape sh = gn_shape(a.f.D);
    return sh.vec == 1 ? gn_bwd_as<Y, G, 1>(a, sh, ctas, s, pdl) : gn_bwd_as<Y, G, 2>(a, sh, ctas, s, pdl);
}

}  // namespace

int gated_norm_bwd_ctas(long long T, int D, bool branch, int sms) {
    const GnShape sh = gn_shape(D);
    return (int)std::max(1LL, std::min<long long>((T + sh.block.y - 1) / sh.block.y,
                                                  (long long)gn_ctas_per_sm(sh, branch ? 512 : 1024) * sms));
}

cudaError_t launch_gated_norm_fwd(const GatedNormArgs& a, cudaStream_t s, bool pdl) {
    if (a.y == nullptr) return gn_fwd<false, false>(a, s, pdl);
    return a.g == nullptr ? gn_fwd<true, false>(a, s, pdl) : gn_fwd<true, true>(a, s, pdl);
}
cudaError_t launch_gated_norm_bwd(const GatedNormBwdArgs& a, int ctas, cudaStream_t s, bool pdl) {
    if (a.f.y == nullptr) return gn_bwd<false, false>(a, ctas, s, pdl);
    return a.f.g == nullptr ? gn_bwd<true, false>(a, ctas, s, pdl) : gn_bwd<true, true>(a, ctas, s, pdl);
}
cudaError_t launch_gated_norm_sum(const GatedNormBwdArgs& a, int parts, float* dgamma_pre, float* dgamma_post,
                                  float* dscale, cudaStream_t s, bool pdl) {
    return launch_ex(gated_norm_sum_kernel, dim3((unsigned)((a.f.D + 31) / 32), a.f.y != nullptr ? 2u : 1u), dim3(1024),
                     0, s, pdl, a.part, parts, a.f.D, a.f.gamma_post, a.f.scale, dgamma_pre, dgamma_post, dscale);
}

}  // namespace lrs

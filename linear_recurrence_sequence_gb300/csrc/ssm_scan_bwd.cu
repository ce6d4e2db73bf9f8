// Backward of the selective state space scan (ssm_scan.cu).
//
// With the cotangent dy' = dy SiLU(gate) of the sum over the states, the adjoint
// of the state runs from the last token to the first:
//   G_t = dy'_t c_t + u_(t+1),  u_t = a_t G_t          (u = 0 at a sequence's first token)
//   dc_t = sum_ch dy'_t h_t          db_t = sum_ch dt_t x_t G_t
//   s1 = sum_n G_t b_t               r_t = u_t h_(t-1)
//   dx = s1 dt + d_skip dy'          ddt = s1 x + sum_n A r,  ddelta = ddt sigmoid(raw)
//   dA = sum_t dt r                  da_log = A dA
//
// Time is cut into chunks as in the forward:
//   rmaps   each chunk but the first from a zero adjoint: what it passes to the
//           chunk before, and the sum of its dt;
//   prefix  the adjoint that reaches each chunk's end (ssm_scan.cu);
//   main    each chunk, eight tokens at a time from the last to the first: the
//           states of the eight tokens again from the state that the forward
//           kept before them, then the adjoint back through them;
//   finish  the sums over chunks and over the CTAs of a token, in a fixed order.
// In main the states before tokens 0, 2, 4, 6 wait in shared memory (16 KB a
// warp), a state before an odd token is formed again from the one before it: a
// store and a load of every state would take more of shared memory's bandwidth
// than the two operations take of the FP32 pipe.  13 multiply-adds and two
// exponentials a (token, channel, state) there, 3 and one in rmaps: bound by the
// FP32 pipe, with the sums across lanes (one shuffle a state) beside it.
#include <algorithm>

#include "ssm.cuh"

namespace lrs {

namespace {

constexpr int kBwdWarps = 4;
constexpr float kLn2 = 0.6931471805599453f;

// dy' = dy SiLU(gate) of 8 channels.
__device__ __forceinline__ void gated(const uint4 qy, const uint4 qz, bool gate, f2x (&dy)[4]) {
    unpack_pairs(qy, dy);
    if (!gate) return;
    f2x z[4];
    unpack_pairs(qz, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float z0, z1;
        up2(z[e], z0, z1);
        dy[e] = mul2(dy[e], mul2(z[e], pk2(ssm_sigmoid(z0), ssm_sigmoid(z1))));
    }
}

struct BwdPlace {
    int b, chunk, group, warp;
    bool on;
};
__device__ __forceinline__ BwdPlace bwd_place(const SsmArgs& a, int chunks, int first) {
    BwdPlace p;
    const long long i = blockIdx.x;
    const int gq = (int)(i % a.ngq);
    const long long r = i / a.ngq;
    p.chunk = first + (int)(r % chunks);
    p.b = (int)(r / chunks);
    p.warp = threadIdx.x >> 5;
    p.group = gq * (blockDim.x >> 5) + p.warp;
    p.on = p.group < a.groups;
    return p;
}

template <int LN>
struct RevTile {
    static constexpr int T = LN == 1 ? 8 : 16;
    using W = SsmWarp<LN>;
    float dt[T][W::CW];
    float dy[T][W::CW];
    float c[T][W::NP];
};

template <int LN>
__global__ void __launch_bounds__(kBwdWarps * 32, 4) ssm_rmaps_kernel(const SsmBwdArgs g) {
    using W = SsmWarp<LN>;
    constexpr int T = RevTile<LN>::T, IT = T / W::RPI;
    extern __shared__ __align__(16) uint8_t buf[];
    pdl_trigger();
    pdl_wait();
    const SsmArgs& a = g.f;
    const int lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN;
    const BwdPlace p = bwd_place(a, a.nchunk - 1, 1);
    if (!p.on) return;
    RevTile<LN>& s = reinterpret_cast<RevTile<LN>*>(buf)[p.warp];
    const int c0 = p.group * W::CW, ch = c0 + lc * kSsmCh;
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL;
    const bool on = c0 + c8 < a.D;
    f2x A[kSsmCh][4], u[kSsmCh][4];
    load_rates<LN>(a.a_log, ch, ln * kSsmSt, a.D, a.N, A);
#pragma unroll
    for (int i = 0; i < kSsmCh; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) u[i][j] = 0ull;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    bool cut = false;
    const int begin = p.chunk * a.chunk, end = min(a.L, begin + a.chunk);
    for (int t0 = begin + (end - 1 - begin) / T * T; t0 >= begin; t0 -= T) {
        const int nt = min(T, end - t0);
        __syncwarp();
        {
            const uint16_t* pd = a.delta.p + (long long)p.b * a.delta.sb + (long long)t0 * a.delta.st + c0 + c8;
            const uint16_t* pz = a.gate.p + (long long)p.b * a.gate.sb + (long long)t0 * a.gate.st + c0 + c8;
            const uint16_t* py = g.dy + ((long long)p.b * a.L + t0) * a.D + c0 + c8;
            uint4 qd[IT], qy[IT], qz[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                qd[i] = qy[i] = qz[i] = make_uint4(0u, 0u, 0u, 0u);
                if (on && r < nt) {
                    qd[i] = __ldg(reinterpret_cast<const uint4*>(pd + (long long)r * a.delta.st));
                    qy[i] = __ldg(reinterpret_cast<const uint4*>(py + (long long)r * a.D));
                    if (a.gate.p != nullptr) qz[i] = __ldg(reinterpret_cast<const uint4*>(pz + (long long)r * a.gate.st));
                }
            }
            f2x bias[4];
            load_pairs(a.delta_bias == nullptr ? nullptr : a.delta_bias + c0 + c8, on, bias);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                f2x d[4], dy[4];
                unpack_pairs(qd[i], d);
                gated(qy[i], qz[i], a.gate.p != nullptr, dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = on && r < nt ? softplus2(add2(d[e], bias[e])) : 0ull;
                store_pairs(&s.dt[r][c8], d);
                store_pairs(&s.dy[r][c8], dy);
            }
        }
        stage_states<LN, T>(a.c, p.b, t0, nt, a.N, &s.c[0][0], lane);
        const uint32_t starts = start_bits(a.reset, (long long)p.b * a.L + t0, nt, lane);
        cut |= starts != 0u;
        __syncwarp();
#pragma unroll 2
        for (int t = T - 1; t >= 0; --t) {
            const float4 dt = *reinterpret_cast<const float4*>(&s.dt[t][lc * kSsmCh]);
            const float4 dy = *reinterpret_cast<const float4*>(&s.dy[t][lc * kSsmCh]);
            const float ds[kSsmCh] = {dt.x, dt.y, dt.z, dt.w}, ys[kSsmCh] = {dy.x, dy.y, dy.z, dy.w};
            f2x c[4];
            read_states(&s.c[t][ln * kSsmSt], c);
#pragma unroll
            for (int i = 0; i < kSsmCh; ++i) {
                const f2x d2 = dup2(ds[i]), y2 = dup2(ys[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float e0, e1;
                    up2(mul2(A[i][j], d2), e0, e1);
                    u[i][j] = mul2(pk2(ex2_approx(e0), ex2_approx(e1)), fma2(y2, c[j], u[i][j]));
                }
            }
            if ((starts >> t) & 1u) {
#pragma unroll
                for (int i = 0; i < kSsmCh; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[i][j] = 0ull;
            }
            sum.x += dt.x;
            sum.y += dt.y;
            sum.z += dt.z;
            sum.w += dt.w;
        }
    }
    const long long slot = ((long long)p.b * a.nchunk + p.chunk) * a.groups + p.group;
    store_tile_state(a.maps + slot * (kSsmVec * 32), lane, u);
    if (cut) sum = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);
    if (ln == 0) *reinterpret_cast<float4*>(a.sums + slot * W::CW + lc * kSsmCh) = sum;
}

constexpr int kBT = kSsmKeep;   // tokens of a tile of the main kernel

template <int LN>
struct BwdTile {
    using W = SsmWarp<LN>;
    float4 h[kBT / 2][kSsmVec][32];   // states before the even tokens
    float dt[kBT][W::CW];             // then s1 dt
    float x[kBT][W::CW];              // then ddt
    float dy[kBT][W::CW];             // dy'
    float y[kBT][W::CW];              // sums c h
    float b[kBT][W::NP];
    float c[kBT][W::NP];
    float red[kBT][2 * W::NP];        // db, dc of the warp's channels
};

// Sums of v[0 .. 7] (four pairs) over the lanes that hold the same states; the
// lanes write theirs to out[8].
template <int LN>
__device__ __forceinline__ void sum_channels(const f2x (&v2)[4], float* out, int lane) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) up2(v2[j], v[2 * j], v[2 * j + 1]);
    int keep = 8;
#pragma unroll
    for (int m = 16; m >= LN; m >>= 1) {
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
    if (LN == 8) {   // two values are left to a lane
        *reinterpret_cast<float2*>(out + (lane >> 4) * 4 + ((lane >> 3) & 1) * 2) = make_float2(v[0], v[1]);
    } else if ((lane & 3 & ~(LN - 1)) == 0) {
        out[(lane >> 4) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1)] = v[0];
    }
}

// a = e^(A dt)
__device__ __forceinline__ f2x decay(f2x A, f2x dt) {
    float e0, e1;
    up2(mul2(A, dt), e0, e1);
    return pk2(ex2_approx(e0), ex2_approx(e1));
}

// One token's adjoint for 8 states of a channel, given a and the state before.
__device__ __forceinline__ void adjoint(f2x y2, f2x k2, f2x d2, const f2x (&A)[4], const f2x (&a)[4], const f2x (&hp)[4],
                                        const f2x (&b)[4], const f2x (&c)[4], f2x (&u)[4], f2x (&db)[4], f2x (&dA)[4],
                                        float& s1, float& s2) {
    f2x p1 = 0ull, p2 = 0ull;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f2x G = fma2(y2, c[j], u[j]);
        p1 = j ? fma2(G, b[j], p1) : mul2(G, b[j]);
        db[j] = fma2(k2, G, db[j]);
        u[j] = mul2(a[j], G);
        const f2x r = mul2(u[j], hp[j]);
        p2 = j ? fma2(A[j], r, p2) : mul2(A[j], r);
        dA[j] = fma2(d2, r, dA[j]);
    }
    float lo, hi;
    up2(p1, lo, hi);
    s1 = lo + hi;
    up2(p2, lo, hi);
    s2 = lo + hi;
}

// Tokens 2 p + 1 and 2 p of a tile.  CUT: a sequence may start at either.
template <int LN, bool CUT>
__device__ __forceinline__ void back_pair(BwdTile<LN>& s, int p, uint32_t starts, int lane, const f2x (&A)[kSsmCh][4],
                                          f2x (&u)[kSsmCh][4], f2x (&dA)[kSsmCh][4]) {
    const int ln = lane % LN, lc = lane / LN;
    const int t0 = 2 * p, t1 = t0 + 1;
    const float4 dt0 = *reinterpret_cast<const float4*>(&s.dt[t0][lc * kSsmCh]);
    const float4 dt1 = *reinterpret_cast<const float4*>(&s.dt[t1][lc * kSsmCh]);
    const float4 x0 = *reinterpret_cast<const float4*>(&s.x[t0][lc * kSsmCh]);
    const float4 x1 = *reinterpret_cast<const float4*>(&s.x[t1][lc * kSsmCh]);
    const float4 y0 = *reinterpret_cast<const float4*>(&s.dy[t0][lc * kSsmCh]);
    const float4 y1 = *reinterpret_cast<const float4*>(&s.dy[t1][lc * kSsmCh]);
    const float d0[4] = {dt0.x, dt0.y, dt0.z, dt0.w}, d1[4] = {dt1.x, dt1.y, dt1.z, dt1.w};
    const float xs0[4] = {x0.x, x0.y, x0.z, x0.w}, xs1[4] = {x1.x, x1.y, x1.z, x1.w};
    const float ys0[4] = {y0.x, y0.y, y0.z, y0.w}, ys1[4] = {y1.x, y1.y, y1.z, y1.w};
    f2x b0[4], b1[4], c0[4], c1[4], db0[4], db1[4];
    read_states(&s.b[t0][ln * kSsmSt], b0);
    read_states(&s.b[t1][ln * kSsmSt], b1);
    read_states(&s.c[t0][ln * kSsmSt], c0);
    read_states(&s.c[t1][ln * kSsmSt], c1);
#pragma unroll
    for (int j = 0; j < 4; ++j) db0[j] = db1[j] = 0ull;
    float dx0[kSsmCh], dx1[kSsmCh], dd0[kSsmCh], dd1[kSsmCh];
    const bool cut0 = CUT && ((starts >> t0) & 1u), cut1 = CUT && ((starts >> t1) & 1u);
#pragma unroll
    for (int i = 0; i < kSsmCh; ++i) {
        const float4 q0 = s.h[p][2 * i][lane], q1 = s.h[p][2 * i + 1][lane];
        f2x hp[4] = {pk2(q0.x, q0.y), pk2(q0.z, q0.w), pk2(q1.x, q1.y), pk2(q1.z, q1.w)}, hq[4], a0[4], a1[4];
        const f2x e0 = dup2(d0[i]), e1 = dup2(d1[i]), k0 = mul2(e0, dup2(xs0[i])), k1 = mul2(e1, dup2(xs1[i]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a0[j] = decay(A[i][j], e0);
            a1[j] = decay(A[i][j], e1);
            if (CUT && cut0) {
                a0[j] = 0ull;
                hp[j] = 0ull;
            }
            hq[j] = fma2(a0[j], hp[j], mul2(k0, b0[j]));
            if (CUT && cut1) {
                a1[j] = 0ull;
                hq[j] = 0ull;
            }
        }
        float s1, s2;
        adjoint(dup2(ys1[i]), k1, e1, A[i], a1, hq, b1, c1, u[i], db1, dA[i], s1, s2);
        dx1[i] = s1 * d1[i];
        dd1[i] = fmaf(s1, xs1[i], kLn2 * s2);
        adjoint(dup2(ys0[i]), k0, e0, A[i], a0, hp, b0, c0, u[i], db0, dA[i], s1, s2);
        dx0[i] = s1 * d0[i];
        dd0[i] = fmaf(s1, xs0[i], kLn2 * s2);
    }
    sum_states<LN>(dx1, lane);
    sum_states<LN>(dd1, lane);
    sum_states<LN>(dx0, lane);
    sum_states<LN>(dd0, lane);
    __syncwarp();   // every lane has read the tokens' dt and x
    put_channels<LN>(s.dt[t1], dx1, lc, ln);
    put_channels<LN>(s.x[t1], dd1, lc, ln);
    put_channels<LN>(s.dt[t0], dx0, lc, ln);
    put_channels<LN>(s.x[t0], dd0, lc, ln);
    sum_channels<LN>(db1, &s.red[t1][ln * kSsmSt], lane);
    sum_channels<LN>(db0, &s.red[t0][ln * kSsmSt], lane);
}

__device__ __forceinline__ void put8(void* p, long long at, bool f32, const f2x (&v)[4]) {
    if (f32)
        store_pairs(static_cast<float*>(p) + at, v);
    else
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(x2bf(v[0]), x2bf(v[1]), x2bf(v[2]), x2bf(v[3]));
}

template <int LN, bool GATE>
__global__ void __launch_bounds__(kBwdWarps * 32, 2) ssm_bwd_kernel(const SsmBwdArgs g) {
    using W = SsmWarp<LN>;
    constexpr int IT = kBT / W::RPI > 0 ? kBT / W::RPI : 1;
    extern __shared__ __align__(16) uint8_t buf[];
    pdl_trigger();
    pdl_wait();
    const SsmArgs& a = g.f;
    const int lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN;
    const BwdPlace p = bwd_place(a, a.nchunk, 0);
    BwdTile<LN>* tiles = reinterpret_cast<BwdTile<LN>*>(buf);
    BwdTile<LN>& s = tiles[p.warp];
    const int c0 = p.group * W::CW, ch = c0 + lc * kSsmCh;
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL;
    const bool on = p.on && c0 + c8 < a.D;
    f2x A[kSsmCh][4], u[kSsmCh][4], dA[kSsmCh][4];
    load_rates<LN>(a.a_log, ch, ln * kSsmSt, a.D, a.N, A);
    const long long slot = ((long long)p.b * a.nchunk + p.chunk) * a.groups + p.group;
    if (a.nchunk > 1 && p.on)
        load_tile_state(a.maps + slot * (kSsmVec * 32), lane, u);
    else
        load_state(a.h0, p.b, ch, ln * kSsmSt, a.D, a.N, u);   // here h0 is the cotangent of the last state
#pragma unroll
    for (int i = 0; i < kSsmCh; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dA[i][j] = 0ull;
    f2x dskip[4] = {0ull, 0ull, 0ull, 0ull}, dbias[4] = {0ull, 0ull, 0ull, 0ull};
    f2x bias[4], skip[4];
    load_pairs(a.delta_bias == nullptr ? nullptr : a.delta_bias + c0 + c8, on, bias);
    load_pairs(a.d_skip == nullptr ? nullptr : a.d_skip + c0 + c8, on, skip);
    const int begin = p.chunk * a.chunk, end = min(a.L, begin + a.chunk);
    const int slots = (a.L + kSsmKeep - 1) / kSsmKeep;
    for (int t0 = begin + (end - 1 - begin) / kBT * kBT; t0 >= begin; t0 -= kBT) {
        const int nt = min(kBT, end - t0);
        const long long row = (long long)p.b * a.L + t0;
        const long long ox = (long long)p.b * a.x.sb + (long long)t0 * a.x.st + c0 + c8;
        const long long od = (long long)p.b * a.delta.sb + (long long)t0 * a.delta.st + c0 + c8;
        const long long oz = (long long)p.b * a.gate.sb + (long long)t0 * a.gate.st + c0 + c8;
        const long long oy = row * a.D + c0 + c8;
        uint32_t starts = 0u;
        if (p.on) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                if (r >= kBT) break;
                const bool in = on && r < nt;
                uint4 qx = make_uint4(0u, 0u, 0u, 0u), qd = qx, qy = qx, qz = qx;
                if (in) {
                    qx = __ldg(reinterpret_cast<const uint4*>(a.x.p + ox + (long long)r * a.x.st));
                    qd = __ldg(reinterpret_cast<const uint4*>(a.delta.p + od + (long long)r * a.delta.st));
                    qy = __ldg(reinterpret_cast<const uint4*>(g.dy + oy + (long long)r * a.D));
                    if (GATE) qz = __ldg(reinterpret_cast<const uint4*>(a.gate.p + oz + (long long)r * a.gate.st));
                }
                f2x x[4], d[4], dy[4];
                unpack_pairs(qx, x);
                unpack_pairs(qd, d);
                gated(qy, qz, GATE, dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[e] = in ? softplus2(add2(d[e], bias[e])) : 0ull;
                    dskip[e] = fma2(dy[e], x[e], dskip[e]);
                }
                store_pairs(&s.dt[r][c8], d);
                store_pairs(&s.x[r][c8], x);
                store_pairs(&s.dy[r][c8], dy);
            }
            stage_states<LN, kBT>(a.b, p.b, t0, nt, a.N, &s.b[0][0], lane);
            stage_states<LN, kBT>(a.c, p.b, t0, nt, a.N, &s.c[0][0], lane);
            starts = start_bits(a.reset, row, nt, lane);
        }
        // the other warps have taken the sums of the tile before
        __syncthreads();
        if (p.on) {
            f2x h[kSsmCh][4];
            load_tile_state(a.keep + (((long long)p.b * slots + t0 / kSsmKeep) * a.groups + p.group) * (kSsmVec * 32), lane, h);
#pragma unroll 2
            for (int t = 0; t < kBT; ++t) {
                if ((t & 1) == 0) store_tile_state(&s.h[t / 2][0][0], lane, h);
                if ((starts >> t) & 1u) {
#pragma unroll
                    for (int i = 0; i < kSsmCh; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) h[i][j] = 0ull;
                }
                const float4 dt = *reinterpret_cast<const float4*>(&s.dt[t][lc * kSsmCh]);
                const float4 x = *reinterpret_cast<const float4*>(&s.x[t][lc * kSsmCh]);
                const float4 dy = *reinterpret_cast<const float4*>(&s.dy[t][lc * kSsmCh]);
                const float ds[4] = {dt.x, dt.y, dt.z, dt.w}, xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {dy.x, dy.y, dy.z, dy.w};
                f2x b[4], c[4], dc[4] = {0ull, 0ull, 0ull, 0ull};
                read_states(&s.b[t][ln * kSsmSt], b);
                if (GATE) read_states(&s.c[t][ln * kSsmSt], c);
                float y[kSsmCh];
#pragma unroll
                for (int i = 0; i < kSsmCh; ++i) {
                    const f2x d2 = dup2(ds[i]), k2 = mul2(d2, dup2(xs[i])), y2 = dup2(ys[i]);
                    f2x acc = 0ull;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h[i][j] = fma2(decay(A[i][j], d2), h[i][j], mul2(k2, b[j]));
                        dc[j] = fma2(y2, h[i][j], dc[j]);
                        if (GATE) acc = j ? fma2(h[i][j], c[j], acc) : mul2(h[i][j], c[j]);
                    }
                    float lo, hi;
                    up2(acc, lo, hi);
                    y[i] = lo + hi;
                }
                if (GATE) {
                    sum_states<LN>(y, lane);
                    put_channels<LN>(s.y[t], y, lc, ln);
                }
                sum_channels<LN>(dc, &s.red[t][W::NP + ln * kSsmSt], lane);
            }
            if (starts == 0u) {
#pragma unroll 1
                for (int q = kBT / 2 - 1; q >= 0; --q) back_pair<LN, false>(s, q, 0u, lane, A, u, dA);
            } else {
#pragma unroll 1
                for (int q = kBT / 2 - 1; q >= 0; --q) back_pair<LN, true>(s, q, starts, lane, A, u, dA);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                if (!on || r >= nt) break;
                f2x v[4], dy[4], t[4];
                read_pairs(&s.dt[r][c8], v);
                read_pairs(&s.dy[r][c8], dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fma2(skip[e], dy[e], v[e]);
                put8(g.dx.p, (long long)p.b * g.dx.sb + (long long)(t0 + r) * g.dx.st + c0 + c8, g.f32, v);
                read_pairs(&s.x[r][c8], v);
                unpack_pairs(__ldg(reinterpret_cast<const uint4*>(a.delta.p + od + (long long)r * a.delta.st)), t);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float r0_, r1_;
                    up2(add2(t[e], bias[e]), r0_, r1_);
                    v[e] = mul2(v[e], pk2(ssm_sigmoid(r0_), ssm_sigmoid(r1_)));
                    dbias[e] = add2(dbias[e], v[e]);
                }
                put8(g.ddelta.p, (long long)p.b * g.ddelta.sb + (long long)(t0 + r) * g.ddelta.st + c0 + c8, g.f32, v);
                if (GATE) {
                    f2x z[4], x[4];
                    read_pairs(&s.y[r][c8], v);
                    unpack_pairs(__ldg(reinterpret_cast<const uint4*>(a.x.p + ox + (long long)r * a.x.st)), x);
                    unpack_pairs(__ldg(reinterpret_cast<const uint4*>(g.dy + oy + (long long)r * a.D)), dy);
                    unpack_pairs(__ldg(reinterpret_cast<const uint4*>(a.gate.p + oz + (long long)r * a.gate.st)), z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float z0, z1;
                        up2(z[e], z0, z1);
                        const f2x sg = pk2(ssm_sigmoid(z0), ssm_sigmoid(z1)), one = dup2(1.f);
                        // SiLU'(z) = s (1 + z (1 - s))
                        const f2x slope = mul2(sg, fma2(z[e], sub2(one, sg), one));
                        v[e] = mul2(mul2(dy[e], fma2(skip[e], x[e], v[e])), slope);
                    }
                    put8(g.dgate.p, (long long)p.b * g.dgate.sb + (long long)(t0 + r) * g.dgate.st + c0 + c8, g.f32, v);
                }
            }
        }
        __syncthreads();
        // db and dc of the CTA's channels, its warps in order
        const int warps = blockDim.x >> 5, live = min(warps, a.groups - (p.group - p.warp));
        const long long gq = blockIdx.x % a.ngq;
        for (int i = threadIdx.x; i < nt * 2 * W::NP; i += blockDim.x) {
            const int t = i / (2 * W::NP), n = i % (2 * W::NP);
            float v = 0.f;
            for (int w = 0; w < live; ++w) v += tiles[w].red[t][n];
            g.dbc[((row + t) * a.ngq + gq) * (2 * W::NP) + n] = v;
        }
    }
    if (!p.on) return;
    const long long part = (long long)p.b * a.nchunk + p.chunk;
    // a part: dA [groups][kSsmVec][32] float4, then the two vectors [2][groups CW]
    float4* out = g.part + part * g.part_len;
    store_tile_state(out + (long long)p.group * (kSsmVec * 32), lane, dA);
    float* vec = reinterpret_cast<float*>(out + (long long)a.groups * (kSsmVec * 32));
    float v[16];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        up2(dskip[e], v[2 * e], v[2 * e + 1]);
        up2(dbias[e], v[8 + 2 * e], v[8 + 2 * e + 1]);
    }
#pragma unroll
    for (int m = W::RL; m < 32; m <<= 1)
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], m);
    if (r0 == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float4* o = reinterpret_cast<float4*>(vec + (long long)w * a.groups * W::CW + c0 + c8);
            o[0] = make_float4(v[8 * w], v[8 * w + 1], v[8 * w + 2], v[8 * w + 3]);
            o[1] = make_float4(v[8 * w + 4], v[8 * w + 5], v[8 * w + 6], v[8 * w + 7]);
        }
    }
    if (p.chunk == 0 && g.dh0 != nullptr) store_state(g.dh0, p.b, ch, ln * kSsmSt, a.D, a.N, u);
}

// The parts of the parameters' gradients joined (the first `columns` CTAs: 32
// float4 columns each, 8 warps with every eighth part), and the CTAs' shares of db, dc.
template <int LN>
__global__ void __launch_bounds__(256) ssm_finish_kernel(const SsmBwdArgs g, int columns) {
    using W = SsmWarp<LN>;
    pdl_trigger();
    pdl_wait();
    const SsmArgs& a = g.f;
    if ((int)blockIdx.x >= columns) {
        const long long n = (long long)a.B * a.L * 2 * W::NP;
        for (long long i = (long long)(blockIdx.x - columns) * 256 + threadIdx.x; i < n;
             i += (long long)(gridDim.x - columns) * 256) {
            const long long row = i / (2 * W::NP);
            const int n2 = (int)(i % (2 * W::NP)), st = n2 % W::NP;
            const float* q = g.dbc + row * a.ngq * (2 * W::NP) + n2;
            float v = 0.f;
            for (int k = 0; k < a.ngq; ++k) v += __ldcg(q + (long long)k * 2 * W::NP);
            if (st >= a.N) continue;
            void* o = n2 < W::NP ? g.db : g.dc;
            if (g.f32)
                static_cast<float*>(o)[row * a.N + st] = v;
            else
                static_cast<__nv_bfloat16*>(o)[row * a.N + st] = __float2bfloat16_rn(v);
        }
        return;
    }
    __shared__ float4 acc[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long col = (long long)blockIdx.x * 32 + lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < g.part_len) {
        const long long parts = (long long)a.B * a.nchunk;
#pragma unroll 4
        for (long long i = w; i < parts; i += 8) {
            const float4 q = __ldcg(g.part + i * g.part_len + col);
            v.x += q.x;
            v.y += q.y;
            v.z += q.z;
            v.w += q.w;
        }
    }
    acc[w][lane] = v;
    __syncthreads();
    if (w != 0 || col >= g.part_len) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        const float4 q = acc[i][lane];
        v.x += q.x;
        v.y += q.y;
        v.z += q.z;
        v.w += q.w;
    }
    const float e[4] = {v.x, v.y, v.z, v.w};
    const long long states = (long long)a.groups * (kSsmVec * 32);
    if (col < states) {
        const int sl = (int)(col & 31), k = (int)(col >> 5) & (kSsmVec - 1);
        const long long grp = col / (kSsmVec * 32);
        const long long c = grp * W::CW + sl / LN * kSsmCh + (k >> 1);
        const int n0 = sl % LN * kSsmSt + 4 * (k & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c < a.D && n0 + j < a.N)
                g.da_log[c * a.N + n0 + j] = -expf(__ldg(a.a_log + c * a.N + n0 + j)) * e[j];
        return;
    }
    const long long at = (col - states) * 4, width = (long long)a.groups * W::CW;
    float* o = at < width ? g.dd_skip : g.ddelta_bias;
    const long long c = at % width;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (o != nullptr && c + j < a.D) o[c + j] = e[j];
}

template <int LN>
cudaError_t bwd_as(const SsmBwdArgs& g, int what, cudaStream_t s, bool pdl) {
    const SsmArgs& a = g.f;
    const SsmSplit w = ssm_split(a.D, a.N);
    const dim3 block((unsigned)w.warps * 32);
    if (what == 0) {
        static std::atomic<bool> allowed[64];
        const size_t smem = w.warps * sizeof(RevTile<LN>), most = kBwdWarps * sizeof(RevTile<LN>);
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_rmaps_kernel<LN>), most, allowed);
        if (e != cudaSuccess) return e;
        return launch_ex(ssm_rmaps_kernel<LN>, dim3((unsigned)((long long)a.B * (a.nchunk - 1) * a.ngq)), block, smem, s, pdl, g);
    }
    if (what == 1) {
        const size_t smem = w.warps * sizeof(BwdTile<LN>), most = kBwdWarps * sizeof(BwdTile<LN>);
        const dim3 grid((unsigned)((long long)a.B * a.nchunk * a.ngq));
        if (a.gate.p != nullptr) {
            static std::atomic<bool> allowed[64];
            const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_bwd_kernel<LN, true>), most, allowed);
            if (e != cudaSuccess) return e;
            return launch_ex(ssm_bwd_kernel<LN, true>, grid, block, smem, s, pdl, g);
        }
        static std::atomic<bool> allowed[64];
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_bwd_kernel<LN, false>), most, allowed);
        if (e != cudaSuccess) return e;
        return launch_ex(ssm_bwd_kernel<LN, false>, grid, block, smem, s, pdl, g);
    }
    const int columns = (int)((g.part_len + 31) / 32);
    const long long n = (long long)a.B * a.L * 2 * SsmWarp<LN>::NP;
    const int rest = (int)std::min<long long>((n + 255) / 256, 152 * 16);
    return launch_ex(ssm_finish_kernel<LN>, dim3((unsigned)(columns + rest)), dim3(256), 0, s, pdl, g, columns);
}
cudaError_t bwd(const SsmBwdArgs& g, int what, cudaStream_t s, bool pdl) {
    switch (ssm_split(g.f.D, g.f.N).lanes) {
        case 1: return bwd_as<1>(g, what, s, pdl);
        case 2: return bwd_as<2>(g, what, s, pdl);
        case 4: return bwd_as<4>(g, what, s, pdl);
        default: return bwd_as<8>(g, what, s, pdl);
    }
}

}  // namespace

cudaError_t launch_ssm_rmaps(const SsmBwdArgs& g, cudaStream_t s, bool pdl) { return bwd(g, 0, s, pdl); }
cudaError_t launch_ssm_bwd(const SsmBwdArgs& g, cudaStream_t s, bool pdl) { return bwd(g, 1, s, pdl); }
cudaError_t launch_ssm_finish(const SsmBwdArgs& g, cudaStream_t s, bool pdl) { return bwd(g, 2, s, pdl); }

}  // namespace lrs

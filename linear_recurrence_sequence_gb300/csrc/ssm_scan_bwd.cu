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
// In main the states before the tile's eight tokens wait in tensor memory, 32 columns a
// token (a lane's 4 x 8 states), so that shared memory (42% busy) keeps to the operands,
// which every lane of a channel reads, and 236 to 255 registers a thread hold the rates, the
// adjoint and dA: 2 CTAs an SM, by tensor memory however few warps they have (2 warps an SM
// where D is one group of channels).  Up to 8 states a warp's tile is 39 KB and a CTA of four
// takes 156: one an SM, though time is cut for two.  13 multiply-adds and two exponentials a
// (token, channel, state) there, 3 and one in rmaps.
//   4 x 4096 x 1024, 16 states: rmaps 65 us, prefix 10, main 272, finish 10.
// Main issues 20 instructions for 32 states, 0.56 a clock and scheduler with 2 warps each:
// 7 of them two-wide FP32 ones, which take the pipe and the register file 2 to 4 clocks, 2.4
// exponentials, 3 of the sums across lanes.  Other forms of main measured there: 4 x 4 states
// a lane (4 CTAs an SM, each operand read twice as often) 299 us, 3 CTAs (168 registers,
// spills) 319, scalar FP32 303, the sums of all eight tokens after the tile 297, 4 tokens
// unrolled 293, one 287; the states written in pairs or fours of columns 269 to 275.
#include <algorithm>

#include "ssm.cuh"
#include "umma.cuh"

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

template <int LN>
struct RevTile {
    static constexpr int T = LN == 1 ? 4 : 8;
    using W = SsmWarp<LN>;
    float bias[W::CW];
    float dt[T][W::CW];
    float dy[T][W::CW];
    float c[T][2 * W::NP];
    uint16_t delta[2][T][W::CW], y[2][T][W::CW], gate[2][T][W::CW], rc[2][T][W::NP];
};

// Where the next tile's operands begin.
struct RevRows {
    const uint16_t *x, *delta, *gate, *dy, *b, *c;
};
__device__ __forceinline__ RevRows rows_from(const SsmBwdArgs& g, int b, int t0, int c0) {
    const SsmArgs& a = g.f;
    return {row_at(a.x, b, t0, c0),  row_at(a.delta, b, t0, c0), row_at(a.gate, b, t0, c0),
            g.dy + ((long long)b * a.L + t0) * a.D + c0, row_at(a.b, b, t0, 0), row_at(a.c, b, t0, 0)};
}
// T tokens back.
template <int T>
__device__ __forceinline__ void move_back(const SsmArgs& a, RevRows& r) {
    r.x -= T * a.x.st;
    r.delta -= T * a.delta.st;
    r.gate -= T * a.gate.st;
    r.dy -= T * (long long)a.D;
    r.b -= T * a.b.st;
    r.c -= T * a.c.st;
}

template <int LN>
__device__ __forceinline__ void ask_reverse(const SsmArgs& a, RevRows& r, int nt, int width, RevTile<LN>& s, int q, int lane) {
    constexpr int T = RevTile<LN>::T;
    ask_rows<LN, T>(r.delta, a.delta.st, nt, width, &s.delta[q][0][0], lane);
    ask_rows<LN, T>(r.dy, a.D, nt, width, &s.y[q][0][0], lane);
    if (a.gate.p != nullptr) ask_rows<LN, T>(r.gate, a.gate.st, nt, width, &s.gate[q][0][0], lane);
    if (a.words) ask_states<LN, T>(r.c, a.c.st, nt, a.N, &s.rc[q][0][0], lane);
    copies_commit();
    move_back<T>(a, r);
}

// One token: u <- e^(A dt) (dy' c + u).
template <int LN>
__device__ __forceinline__ void retreat(const RevTile<LN>& s, int t, int lc, int ln, const SsmStates& A, SsmStates& u,
                                        f2x (&dt)[2]) {
    f2x dy[2];
    read_channels(&s.dt[t][lc * kSsmCh], dt);
    read_channels(&s.dy[t][lc * kSsmCh], dy);
#pragma unroll
    for (int j = 0; j < kSsmSt; j += 2) {
        f2x c[2];
        read_twice(&s.c[t][state_at<LN>(ln, j)], c[0], c[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) u[j + e][i] = mul2(decay(A[j + e][i], dt[i]), fma2(dy[i], c[e], u[j + e][i]));
    }
}

template <int LN>
__global__ void __launch_bounds__(kBwdWarps * 32, 4) ssm_rmaps_kernel(const SsmBwdArgs g) {
    using W = SsmWarp<LN>;
    constexpr int T = RevTile<LN>::T, IT = (T + W::RPI - 1) / W::RPI;
    extern __shared__ __align__(16) uint8_t buf[];
    pdl_wait();
    const SsmArgs& a = g.f;
    const int lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN;
    const SsmPlace p = place(a, a.nchunk - 1, 1);
    if (!p.on) return;
    RevTile<LN>& s = reinterpret_cast<RevTile<LN>*>(buf)[p.warp];
    const int c0 = p.group * W::CW, ch = c0 + lc * kSsmCh;
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL;
    SsmStates A, u;
    load_rates(a.a_log, a.rate_quads, ch, ln * kSsmSt, a.D, a.N, A);
    clear_states(u);
    f2x sum[2] = {0ull, 0ull};
    bool cut = false;
    // part k of the main kernel's chunk: a.chunk tokens, what is left for the last
    const int part = p.chunk % g.per, chunk0 = p.chunk / g.per * g.chunk, begin = chunk0 + part * a.chunk;
    const int end = min(a.L, part == g.per - 1 ? chunk0 + g.chunk : begin + a.chunk);
    const int last = begin + (end - 1 - begin) / T * T;
    stage_bias<LN>(a.delta_bias, c0, a.D, s.bias, lane);
    RevRows rows = rows_from(g, p.b, last, c0);
    ask_reverse<LN>(a, rows, end - last, a.D - c0, s, 0, lane);
    for (int t0 = last, q = 0; t0 >= begin; t0 -= T, q ^= 1) {
        const int nt = min(T, end - t0);
        const uint32_t starts = start_bits(a.reset, (long long)p.b * a.L + t0, nt, lane);
        copies_wait();
        __syncwarp();
        f2x bias[4];
        read_pairs(&s.bias[c8], bias);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = r0 + i * W::RPI;
            if (T % W::RPI != 0 && r >= T) break;
            f2x d[4], dy[4];
            unpack_pairs(*reinterpret_cast<const uint4*>(&s.delta[q][r][c8]), d);
            gated(*reinterpret_cast<const uint4*>(&s.y[q][r][c8]), *reinterpret_cast<const uint4*>(&s.gate[q][r][c8]),
                  a.gate.p != nullptr, dy);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = softplus2(add2(d[e], bias[e]));
            store_pairs(&s.dt[r][c8], d);
            store_pairs(&s.dy[r][c8], dy);
        }
        if (nt < T) {   // dy of a token past the end is zero
            const f2x none[4] = {0ull, 0ull, 0ull, 0ull};
            for (int r = r0; r < T; r += W::RPI)
                if (r >= nt) store_pairs(&s.dt[r][c8], none);
        }
        stage_states<LN, T>(row_at(a.c, p.b, t0, 0), a.c.st, a.words, nt, a.N, &s.rc[q][0][0], &s.c[0][0], lane);
        __syncwarp();
        if (t0 > begin) ask_reverse<LN>(a, rows, T, a.D - c0, s, q ^ 1, lane);
        if (starts == 0u) {
#pragma unroll
            for (int t = T - 1; t >= 0; --t) {
                f2x dt[2];
                retreat<LN>(s, t, lc, ln, A, u, dt);
                sum[0] = add2(sum[0], dt[0]);
                sum[1] = add2(sum[1], dt[1]);
            }
            continue;
        }
        cut = true;
#pragma unroll 1
        for (int t = T - 1; t >= 0; --t) {
            f2x dt[2];
            retreat<LN>(s, t, lc, ln, A, u, dt);
            if ((starts >> t) & 1u) clear_states(u);
        }
    }
    pdl_trigger();
    const long long slot = ((long long)p.b * a.nchunk + p.chunk) * a.groups + p.group;
    store_tile_state(a.maps + slot * (kSsmVec * 32), lane, u);
    float4 o;
    up2(sum[0], o.x, o.y);
    up2(sum[1], o.z, o.w);
    if (cut) o = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);
    if (ln == 0) *reinterpret_cast<float4*>(a.sums + slot * W::CW + lc * kSsmCh) = o;
}

constexpr int kBT = kSsmKeep;   // tokens of a tile of the main kernel
constexpr int kBwdTmem = 32 * kBT;   // tensor-memory columns of a CTA

template <int LN>
struct BwdTile {
    using W = SsmWarp<LN>;
    float4 kept[kSsmVec][32];         // the state before the tile
    float dt[kBT][W::CW];
    float k[kBT][W::CW];              // dt x, then sum G b
    float dy[kBT][W::CW];             // dy'
    float y[kBT][W::CW];              // sums c h, then sum A r
    float b[kBT][2 * W::NP];
    float c[kBT][2 * W::NP];
    float red[kBT][2 * W::NP];        // db, dc of the warp's channels
    float bias[W::CW], skip[W::CW];
    uint16_t x[2][kBT][W::CW], delta[2][kBT][W::CW], dys[2][kBT][W::CW], gate[2][kBT][W::CW];
    uint16_t rb[2][kBT][W::NP], rc[2][kBT][W::NP];
};

template <int LN, bool GATE>
__device__ __forceinline__ void ask_back(const SsmArgs& a, const float4* kept, RevRows& r, int nt, int width, BwdTile<LN>& s, int q,
                                         int lane) {
#pragma unroll
    for (int k = 0; k < kSsmVec; ++k) copy16(&s.kept[k][lane], kept + k * 32 + lane, true);
    ask_rows<LN, kBT>(r.x, a.x.st, nt, width, &s.x[q][0][0], lane);
    ask_rows<LN, kBT>(r.delta, a.delta.st, nt, width, &s.delta[q][0][0], lane);
    ask_rows<LN, kBT>(r.dy, a.D, nt, width, &s.dys[q][0][0], lane);
    if (GATE) ask_rows<LN, kBT>(r.gate, a.gate.st, nt, width, &s.gate[q][0][0], lane);
    if (a.words) {
        ask_states<LN, kBT>(r.b, a.b.st, nt, a.N, &s.rb[q][0][0], lane);
        ask_states<LN, kBT>(r.c, a.c.st, nt, a.N, &s.rc[q][0][0], lane);
    }
    copies_commit();
    move_back<kBT>(a, r);
}

// Sums of v[0 .. 7] over the lanes that hold the same states; the lanes write
// theirs to out[8].
template <int LN>
__device__ __forceinline__ void sum_channels(float (&v)[kSsmSt], float* out, int lane) {
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

// A lane's states into 32 columns of tensor memory.
__device__ __forceinline__ void states_to_tmem(uint32_t at, const SsmStates& h) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float lo, hi;
        up2(h[i / 2][i % 2], lo, hi);
        r[2 * i] = __float_as_uint(lo);
        r[2 * i + 1] = __float_as_uint(hi);
    }
    tmem_st32(at, r);
}
__device__ __forceinline__ float both_of(f2x v) {
    float lo, hi;
    up2(v, lo, hi);
    return lo + hi;
}

// One token's state, the one before it left at `at`; dc, and (GATE) the sums c h.
template <int LN, bool GATE>
__device__ __forceinline__ void forth(BwdTile<LN>& s, int t, uint32_t at, int lane, const SsmStates& A, SsmStates& h) {
    const int ln = lane % LN, lc = lane / LN;
    states_to_tmem(at, h);
    f2x dt[2], k[2], dy[2], y2[2];
    read_channels(&s.dt[t][lc * kSsmCh], dt);
    read_channels(&s.k[t][lc * kSsmCh], k);
    read_channels(&s.dy[t][lc * kSsmCh], dy);
    float dc[kSsmSt], y[kSsmCh];
#pragma unroll
    for (int j = 0; j < kSsmSt; j += 2) {
        f2x b[2], c[2];
        read_twice(&s.b[t][state_at<LN>(ln, j)], b[0], b[1]);
        if (GATE) read_twice(&s.c[t][state_at<LN>(ln, j)], c[0], c[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f2x d = 0ull;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                h[j + e][i] = fma2(decay(A[j + e][i], dt[i]), h[j + e][i], mul2(k[i], b[e]));
                d = i ? fma2(dy[i], h[j + e][i], d) : mul2(dy[i], h[j + e][i]);
                if (GATE) y2[i] = j + e ? fma2(h[j + e][i], c[e], y2[i]) : mul2(h[j + e][i], c[e]);
            }
            dc[j + e] = both_of(d);
        }
    }
    if (GATE) {
        sum_states<LN>(y2, y, lane);
        put_channels<LN>(s.y[t], y, lc, ln);
    }
    sum_channels<LN>(dc, &s.red[t][SsmWarp<LN>::NP + ln * kSsmSt], lane);
}

// One token's adjoint; `at`: where the state before it waits.
template <int LN>
__device__ __forceinline__ void back(BwdTile<LN>& s, int t, uint32_t at, int lane, const SsmStates& A, SsmStates& u,
                                     SsmStates& dA) {
    const int ln = lane % LN, lc = lane / LN;
    uint32_t hp[32];
    tmem_ld32(at, hp);
    f2x dt[2], k[2], dy[2], p1[2], p2[2];
    read_channels(&s.dt[t][lc * kSsmCh], dt);
    read_channels(&s.k[t][lc * kSsmCh], k);
    read_channels(&s.dy[t][lc * kSsmCh], dy);
    float db[kSsmSt], s1[kSsmCh], s2[kSsmCh];
#pragma unroll
    for (int j = 0; j < kSsmSt; j += 2) {
        f2x b[2], c[2];
        read_twice(&s.b[t][state_at<LN>(ln, j)], b[0], b[1]);
        read_twice(&s.c[t][state_at<LN>(ln, j)], c[0], c[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f2x d = 0ull;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f2x G = fma2(dy[i], c[e], u[j + e][i]);
                p1[i] = j + e ? fma2(G, b[e], p1[i]) : mul2(G, b[e]);
                d = i ? fma2(k[i], G, d) : mul2(k[i], G);
                u[j + e][i] = mul2(decay(A[j + e][i], dt[i]), G);
            }
            db[j + e] = both_of(d);
        }
    }
    tmem_ld32_wait(hp);
#pragma unroll
    for (int j = 0; j < kSsmSt; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at_ = 4 * j + 2 * i;
            const f2x r = mul2(u[j][i], pk2(__uint_as_float(hp[at_]), __uint_as_float(hp[at_ + 1])));
            p2[i] = j ? fma2(A[j][i], r, p2[i]) : mul2(A[j][i], r);
            dA[j][i] = fma2(dt[i], r, dA[j][i]);
        }
    sum_states<LN>(p1, s1, lane);
    sum_states<LN>(p2, s2, lane);
    // (every lane of a channel has read the token's dt x before it takes part in the sum)
    put_channels<LN>(s.k[t], s1, lc, ln);
    put_channels<LN>(s.y[t], s2, lc, ln);
    sum_channels<LN>(db, &s.red[t][ln * kSsmSt], lane);
}

__device__ __forceinline__ void put8(void* p, long long at, bool f32, const f2x (&v)[4]) {
    if (f32)
        put_pairs(static_cast<float*>(p) + at, v);
    else
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(x2bf(v[0]), x2bf(v[1]), x2bf(v[2]), x2bf(v[3]));
}

template <int LN, bool GATE>
__global__ void __launch_bounds__(kBwdWarps * 32, 2) ssm_bwd_kernel(const SsmBwdArgs g) {
    using W = SsmWarp<LN>;
    constexpr int IT = (kBT + W::RPI - 1) / W::RPI;
    extern __shared__ __align__(16) uint8_t buf[];
    __shared__ uint32_t s_tmem;
    pdl_wait();
    if (threadIdx.x < 32) tmem_alloc(&s_tmem, kBwdTmem);   // not before the wait: see umma.cuh
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const SsmArgs& a = g.f;
    const int lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN;
    const SsmPlace p = place(a, g.nchunk, 0);
    BwdTile<LN>* tiles = reinterpret_cast<BwdTile<LN>*>(buf);
    BwdTile<LN>& s = tiles[p.warp];
    const uint32_t tmem = s_tmem + ((uint32_t)p.warp << 21);   // the warp's 32 lanes
    const int c0 = p.group * W::CW, ch = c0 + lc * kSsmCh;
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL;
    const bool on = p.on && c0 + c8 < a.D;
    SsmStates A, u, dA;
    // (zeros where they need not be: for 9 to 16 states the compiler then keeps to 236 registers, else 255 and spills,
    // 1 x 8192 x 2560 backward 437 us against 433)
    load_rates<LN == 2>(a.a_log, a.rate_quads, ch, ln * kSsmSt, a.D, a.N, A);
    // the chunk ends where the last of its maps does
    const long long slot = ((long long)p.b * a.nchunk + min((p.chunk + 1) * g.per, a.nchunk) - 1) * a.groups + p.group;
    if (a.nchunk > 1 && p.on)
        load_tile_state(a.maps + slot * (kSsmVec * 32), lane, u);
    else
        load_state(a.h0, a.quads, p.b, ch, ln * kSsmSt, a.D, a.N, u);   // here h0 is the cotangent of the last state
    clear_states(dA);
    f2x dskip[4] = {0ull, 0ull, 0ull, 0ull}, dbias[4] = {0ull, 0ull, 0ull, 0ull};
    const int begin = p.chunk * g.chunk, end = min(a.L, begin + g.chunk);
    const int last = begin + (end - 1 - begin) / kBT * kBT;
    const long long stride = (long long)a.groups * (kSsmVec * 32);   // of the kept states, a tile back
    const float4* kept = a.keep + ((long long)p.b * ((a.L + kBT - 1) / kBT) + last / kBT) * stride + (long long)p.group * (kSsmVec * 32);
    stage_bias<LN>(a.delta_bias, c0, a.D, s.bias, lane);
    stage_bias<LN>(a.d_skip, c0, a.D, s.skip, lane);
    RevRows rows = rows_from(g, p.b, last, c0);
    if (p.on) ask_back<LN, GATE>(a, kept, rows, end - last, a.D - c0, s, 0, lane);
    for (int t0 = last, q = 0; t0 >= begin; t0 -= kBT, q ^= 1, kept -= stride) {
        const int nt = min(kBT, end - t0);
        const long long row = (long long)p.b * a.L + t0;
        uint32_t starts = 0u;
        if (p.on) {
            starts = start_bits(a.reset, row, nt, lane);
            copies_wait();
            __syncwarp();
            f2x bias[4];
            read_pairs(&s.bias[c8], bias);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                if (kBT % W::RPI != 0 && r >= kBT) break;
                f2x x[4], d[4], dy[4];
                unpack_pairs(*reinterpret_cast<const uint4*>(&s.x[q][r][c8]), x);
                unpack_pairs(*reinterpret_cast<const uint4*>(&s.delta[q][r][c8]), d);
                gated(*reinterpret_cast<const uint4*>(&s.dys[q][r][c8]), *reinterpret_cast<const uint4*>(&s.gate[q][r][c8]), GATE,
                      dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[e] = softplus2(add2(d[e], bias[e]));
                    dskip[e] = fma2(dy[e], x[e], dskip[e]);
                    x[e] = mul2(d[e], x[e]);
                }
                store_pairs(&s.dt[r][c8], d);
                store_pairs(&s.k[r][c8], x);
                store_pairs(&s.dy[r][c8], dy);
            }
            if (nt < kBT) {   // x and dy of a token past the end are zero
                const f2x none[4] = {0ull, 0ull, 0ull, 0ull};
                for (int r = r0; r < kBT; r += W::RPI)
                    if (r >= nt) store_pairs(&s.dt[r][c8], none);
            }
            stage_states<LN, kBT>(row_at(a.b, p.b, t0, 0), a.b.st, a.words, nt, a.N, &s.rb[q][0][0], &s.b[0][0], lane);
            stage_states<LN, kBT>(row_at(a.c, p.b, t0, 0), a.c.st, a.words, nt, a.N, &s.rc[q][0][0], &s.c[0][0], lane);
        }
        // the other warps have taken the sums of the tile before
        __syncthreads();
        if (p.on) {
            SsmStates h;
#pragma unroll
            for (int k = 0; k < kSsmVec; ++k) {
                const float4 v = s.kept[k][lane];
                h[k][0] = pk2(v.x, v.y);
                h[k][1] = pk2(v.z, v.w);
            }
            if (starts == 0u) {
#pragma unroll 2
                for (int t = 0; t < kBT; ++t) forth<LN, GATE>(s, t, tmem + t * 32, lane, A, h);
            } else {
#pragma unroll 1
                for (int t = 0; t < kBT; ++t) {
                    if ((starts >> t) & 1u) clear_states(h);
                    forth<LN, GATE>(s, t, tmem + t * 32, lane, A, h);
                }
            }
            tmem_st_wait();
            __syncwarp();
            if (t0 > begin) ask_back<LN, GATE>(a, kept - stride, rows, kBT, a.D - c0, s, q ^ 1, lane);
            f2x skip[4];
            read_pairs(&s.skip[c8], skip);
            if (GATE) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int r = r0 + i * W::RPI;
                    if (!on || r >= nt) break;
                    f2x v[4], x[4], dy[4], z[4];
                    read_pairs(&s.y[r][c8], v);
                    unpack_pairs(*reinterpret_cast<const uint4*>(&s.x[q][r][c8]), x);
                    unpack_pairs(*reinterpret_cast<const uint4*>(&s.dys[q][r][c8]), dy);
                    unpack_pairs(*reinterpret_cast<const uint4*>(&s.gate[q][r][c8]), z);
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
                __syncwarp();
            }
            if (starts == 0u) {
#pragma unroll 2
                for (int t = kBT - 1; t >= 0; --t) back<LN>(s, t, tmem + t * 32, lane, A, u, dA);
            } else {
#pragma unroll 1
                for (int t = kBT - 1; t >= 0; --t) {
                    back<LN>(s, t, tmem + t * 32, lane, A, u, dA);
                    // nothing goes past a start (the state before it waits as zeros)
                    if ((starts >> t) & 1u) clear_states(u);
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                if (!on || r >= nt) break;
                f2x v[4], s1[4], t[4], bias[4];
                read_pairs(&s.k[r][c8], s1);
                read_pairs(&s.dt[r][c8], t);
                read_pairs(&s.dy[r][c8], v);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fma2(s1[e], t[e], mul2(skip[e], v[e]));
                put8(g.dx.p, (long long)p.b * g.dx.sb + (long long)(t0 + r) * g.dx.st + c0 + c8, g.f32, v);
                read_pairs(&s.y[r][c8], v);
                unpack_pairs(*reinterpret_cast<const uint4*>(&s.x[q][r][c8]), t);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = fma2(s1[e], t[e], mul2(dup2(kLn2), v[e]));
                unpack_pairs(*reinterpret_cast<const uint4*>(&s.delta[q][r][c8]), t);
                read_pairs(&s.bias[c8], bias);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float w0, w1;
                    up2(add2(t[e], bias[e]), w0, w1);
                    v[e] = mul2(v[e], pk2(ssm_sigmoid(w0), ssm_sigmoid(w1)));
                    dbias[e] = add2(dbias[e], v[e]);
                }
                put8(g.ddelta.p, (long long)p.b * g.ddelta.sb + (long long)(t0 + r) * g.ddelta.st + c0 + c8, g.f32, v);
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
    // late, as in ssm_maps_kernel
    pdl_trigger();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (threadIdx.x < 32) tmem_dealloc(s_tmem, kBwdTmem);
    if (!p.on) return;
    const long long part = (long long)p.b * g.nchunk + p.chunk;
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
    if (p.chunk == 0 && g.dh0 != nullptr) store_state(g.dh0, a.quads, p.b, ch, ln * kSsmSt, a.D, a.N, u);
}

// The parts of the parameters' gradients joined (the first `columns` CTAs: 32
// float4 columns each, 8 warps with every eighth part), and the CTAs' shares of db, dc.
template <int LN>
__global__ void __launch_bounds__(256) ssm_finish_kernel(const SsmBwdArgs g, int columns) {
    using W = SsmWarp<LN>;
    pdl_wait();   // no early trigger: the next call's CTAs would take these ones' places
    const SsmArgs& a = g.f;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;
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
        const long long parts = (long long)a.B * g.nchunk;
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
        const long long c = grp * W::CW + sl / LN * kSsmCh;
        const int n = sl % LN * kSsmSt + k;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < a.D && n < a.N) g.da_log[(c + j) * a.N + n] = finite_rate(-expf(__ldg(a.a_log + (c + j) * a.N + n))) * e[j];
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
        const dim3 grid((unsigned)((long long)a.B * g.nchunk * a.ngq));
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

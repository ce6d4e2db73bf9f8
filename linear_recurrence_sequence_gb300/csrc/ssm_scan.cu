// The selective state space scan, forward and one token at a time.
//
//   dt_t = softplus(delta_t + delta_bias),  a_tn = e^(-e^a_log_n dt_t)
//   h_tn = a_tn h_(t-1)n + dt_t x_t b_tn          (a channel's N states; a = 0 at a sequence's first token)
//   y_t  = (sum_n c_tn h_tn + d_skip x_t) SiLU(gate_t)
//
// One exponential and four multiply-adds a (token, channel, state): at N = 16 a
// value of x brings 16 of them, so the SFU (32 ex2 a clock and SM) and the FP32
// pipe (128 operations) bound it both, above the streams' time at HBM speed.
//
// The recurrence runs through time in registers (ssm.cuh: 4 channels x 8 states
// a lane).  Time is cut into chunks so that every SM has its 16 warps:
//   maps    each chunk but the last from a zero state: its end state, and the
//           sum of its dt, which gives what it keeps of the state before
//           (a product of exponentials is one exponential);
//   prefix  the entry state of every chunk, in place;
//   replay  each chunk again from its entry state, with the outputs.
// The maps cost nearly as much as the replay, so where batch and channels alone
// give enough warps (fewer than three chunks would fit) the replay runs alone.
// A warp stages its own operands for 4 or 8 tokens: x, delta as BF16 rows (128
// bytes of a row at N = 16), dt and dt x as FP32 in shared memory, from where
// the lanes that share a channel read them; the next tokens' rows are copied
// meanwhile.  No barrier between warps.
//   4 x 4096 x 1024, 16 states: maps 59 us (SFU 54%, FP32 pipe 51%), prefix 10, replay
//   88 with the states that the backward needs (FP32 pipe 47%, shared memory 48%); the
//   rest are the two-wide FP32 instructions' register reads and the staging.
//   1 x 8192 x 2560: 76, 12 and 106 us.
#include <algorithm>
#include <cmath>

#include "ssm.cuh"

namespace lrs {

namespace {

constexpr int kSsmWarps = 4;       // of a CTA, at most
constexpr int kSsmCtas = 4;        // resident per SM: 128 registers a thread
constexpr int kSsmSms = 152;

// A warp's share of shared memory: the tile that it goes through, and the next
// one's operands as they lie in memory, which arrive meanwhile.  Y: with what
// only the outputs need.
template <int LN, bool Y>
struct FwdTile {
    // tokens: what leaves an SM four CTAs' room (64 states, 4 x 4096 x 256: 8 tokens 183 us, 4 tokens 169)
    static constexpr int T = LN == 1 || LN == 8 ? 4 : 8;
    using W = SsmWarp<LN>;
    float bias[W::CW];
    float dt[T][W::CW];    // then the sums over the states
    float k[T][W::CW];
    float b[T][2 * W::NP];
    float c[Y ? T : 1][Y ? 2 * W::NP : 4];
    uint16_t x[2][T][W::CW], delta[2][T][W::CW];
    uint16_t gate[Y ? 2 : 1][Y ? T : 1][Y ? W::CW : 8];
    uint16_t rb[2][T][W::NP];
    uint16_t rc[Y ? 2 : 1][Y ? T : 1][Y ? W::NP : 8];
};

// Where the next tile's operands begin.
struct FwdRows {
    const uint16_t *x, *delta, *gate, *b, *c;
};
__device__ __forceinline__ FwdRows rows_from(const SsmArgs& a, int b, int t0, int c0) {
    return {row_at(a.x, b, t0, c0), row_at(a.delta, b, t0, c0), row_at(a.gate, b, t0, c0), row_at(a.b, b, t0, 0),
            row_at(a.c, b, t0, 0)};
}
// Asks for the operands of nt tokens, and moves on.
template <int LN, bool Y>
__device__ __forceinline__ void ask_tile(const SsmArgs& a, FwdRows& r, int nt, int width, FwdTile<LN, Y>& s, int q, int lane) {
    constexpr int T = FwdTile<LN, Y>::T;
    ask_rows<LN, T>(r.x, a.x.st, nt, width, &s.x[q][0][0], lane);
    ask_rows<LN, T>(r.delta, a.delta.st, nt, width, &s.delta[q][0][0], lane);
    if (Y && a.gate.p != nullptr) ask_rows<LN, T>(r.gate, a.gate.st, nt, width, &s.gate[Y ? q : 0][0][0], lane);
    if (a.words) {
        ask_states<LN, T>(r.b, a.b.st, nt, a.N, &s.rb[q][0][0], lane);
        if (Y) ask_states<LN, T>(r.c, a.c.st, nt, a.N, &s.rc[Y ? q : 0][0][0], lane);
    }
    copies_commit();
    r.x += T * a.x.st;
    r.delta += T * a.delta.st;
    if (Y) r.gate += T * a.gate.st;
    r.b += T * a.b.st;
    if (Y) r.c += T * a.c.st;
}

// dt and dt x of nt tokens, b and c in FP32.
template <int LN, bool Y>
__device__ __forceinline__ void stage_tile(const SsmArgs& a, int b, int c0, int t0, int nt, FwdTile<LN, Y>& s, int q, int lane) {
    using W = SsmWarp<LN>;
    constexpr int T = FwdTile<LN, Y>::T, IT = (T + W::RPI - 1) / W::RPI;
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL;
    f2x bias[4];
    read_pairs(&s.bias[c8], bias);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = r0 + i * W::RPI;
        if (T % W::RPI != 0 && r >= T) break;
        f2x x[4], d[4];
        unpack_pairs(*reinterpret_cast<const uint4*>(&s.x[q][r][c8]), x);
        unpack_pairs(*reinterpret_cast<const uint4*>(&s.delta[q][r][c8]), d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            d[e] = softplus2(add2(d[e], bias[e]));
            x[e] = mul2(d[e], x[e]);
        }
        store_pairs(&s.dt[r][c8], d);
        store_pairs(&s.k[r][c8], x);
    }
    if (nt < T) {   // a token past the end keeps the state and adds nothing
        const f2x none[4] = {0ull, 0ull, 0ull, 0ull};
        for (int r = r0; r < T; r += W::RPI)
            if (r >= nt) {
                store_pairs(&s.dt[r][c8], none);
                store_pairs(&s.k[r][c8], none);
            }
    }
    stage_states<LN, T>(row_at(a.b, b, t0, 0), a.b.st, a.words, nt, a.N, &s.rb[q][0][0], &s.b[0][0], lane);
    if (Y) stage_states<LN, T>(row_at(a.c, b, t0, 0), a.c.st, a.words, nt, a.N, &s.rc[Y ? q : 0][0][0], &s.c[0][0], lane);
}

// One token: h <- e^(A dt) h + k b, and (Y) the sums of c h.
template <int LN, bool Y>
__device__ __forceinline__ void advance(const FwdTile<LN, Y>& s, int t, int lc, int ln, const SsmStates& A, SsmStates& h,
                                        f2x (&y)[2], f2x (&dt)[2]) {
    f2x k[2];
    read_channels(&s.dt[t][lc * kSsmCh], dt);
    read_channels(&s.k[t][lc * kSsmCh], k);
#pragma unroll
    for (int j = 0; j < kSsmSt; j += 2) {
        f2x b[2], c[2];
        read_twice(&s.b[t][state_at<LN>(ln, j)], b[0], b[1]);
        if (Y) read_twice(&s.c[t][state_at<LN>(ln, j)], c[0], c[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                h[j + e][i] = fma2(decay(A[j + e][i], dt[i]), h[j + e][i], mul2(k[i], b[e]));
                if (Y) y[i] = j + e ? fma2(h[j + e][i], c[e], y[i]) : mul2(h[j + e][i], c[e]);
            }
    }
}

template <int LN>
__global__ void __launch_bounds__(kSsmWarps * 32, kSsmCtas) ssm_maps_kernel(const SsmArgs a) {
    using W = SsmWarp<LN>;
    constexpr int T = FwdTile<LN, false>::T;
    extern __shared__ __align__(16) uint8_t buf[];
    pdl_wait();
    const int lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN;
    const SsmPlace p = place(a, a.nchunk - 1, 0);
    if (!p.on) return;
    FwdTile<LN, false>& s = reinterpret_cast<FwdTile<LN, false>*>(buf)[p.warp];
    const int c0 = p.group * W::CW, ch = c0 + lc * kSsmCh;
    SsmStates A, h;
    load_rates(a.a_log, a.rate_quads, ch, ln * kSsmSt, a.D, a.N, A);
    clear_states(h);
    f2x sum[2] = {0ull, 0ull};
    bool cut = false;
    const int begin = p.chunk * a.chunk, end = min(a.L, begin + a.chunk);
    stage_bias<LN>(a.delta_bias, c0, a.D, s.bias, lane);
    FwdRows rows = rows_from(a, p.b, begin, c0);
    ask_tile<LN, false>(a, rows, min(T, end - begin), a.D - c0, s, 0, lane);
    for (int t0 = begin, q = 0; t0 < end; t0 += T, q ^= 1) {
        const int nt = min(T, end - t0);
        const uint32_t starts = start_bits(a.reset, (long long)p.b * a.L + t0, nt, lane);
        copies_wait();
        __syncwarp();
        stage_tile<LN, false>(a, p.b, c0, t0, nt, s, q, lane);
        __syncwarp();
        if (t0 + T < end) ask_tile<LN, false>(a, rows, min(T, end - t0 - T), a.D - c0, s, q ^ 1, lane);
        // (a test for starts in the loop would keep a token's loads from moving ahead of the one before it)
        if (starts == 0u) {
#pragma unroll
            for (int t = 0; t < T; ++t) {
                f2x y[2], dt[2];
                advance<LN, false>(s, t, lc, ln, A, h, y, dt);
                sum[0] = add2(sum[0], dt[0]);
                sum[1] = add2(sum[1], dt[1]);
            }
            continue;
        }
        cut = true;   // what the state was before is of no matter, nor is the sum
#pragma unroll 1
        for (int t = 0; t < T; ++t) {
            if ((starts >> t) & 1u) clear_states(h);
            f2x y[2], dt[2];
            advance<LN, false>(s, t, lc, ln, A, h, y, dt);
        }
    }
    // the next kernel's CTAs may come now: come at the start, they took the places of this one's on some SMs
    // (4 x 4096 x 1024 forward + backward 608 us, so 543)
    pdl_trigger();
    const long long slot = ((long long)p.b * a.nchunk + p.chunk) * a.groups + p.group;
    store_tile_state(a.maps + slot * (kSsmVec * 32), lane, h);
    // an infinite sum: nothing is kept
    float4 o;
    up2(sum[0], o.x, o.y);
    up2(sum[1], o.z, o.w);
    if (cut) o = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);
    if (ln == 0) *reinterpret_cast<float4*>(a.sums + slot * W::CW + lc * kSsmCh) = o;
}

// Entry states of the chunks, in place of their end states: one float4 of a
// warp's states a thread.  Backward (REV): the adjoints that reach a chunk's
// end, from the last chunk to the first.  Bound by the loads' latency: CTAs of a warp,
// on as many SMs, and 24 chunks asked for at a time (1 x 32768 x 8, 286 chunks: 256
// threads and 8 chunks 103 us forward, 32 and 24 88; 32 chunks do not fit the registers).
constexpr int kPrefixThreads = 32;
template <int LN, bool REV>
__global__ void __launch_bounds__(kPrefixThreads) ssm_prefix_kernel(const SsmArgs a) {
    using W = SsmWarp<LN>;
    pdl_wait();
    const long long i = (long long)blockIdx.x * kPrefixThreads + threadIdx.x;
    const int lane = (int)(i & 31), k = (int)(i >> 5) & (kSsmVec - 1);
    const long long bg = i / (32 * kSsmVec);
    const int g = (int)(bg % a.groups);
    const long long b = bg / a.groups;
    if (b >= a.B) return;
    const int cw = lane / LN * kSsmCh, c = g * W::CW + cw, n = lane % LN * kSsmSt + k;
    float A[4], h[4];
    const float* start = a.h0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool on = c + e < a.D && n < a.N;
        A[e] = on ? ssm_rate(__ldg(a.a_log + (long long)(c + e) * a.N + n)) : 0.f;
        h[e] = on && start != nullptr ? __ldg(start + (b * a.D + c + e) * a.N + n) : 0.f;
    }
    // forward: chunk i's entry from chunk i - 1's; the last chunk has no map of its own
    const long long step = (REV ? -1 : 1) * (long long)a.groups;
    const long long first = (b * a.nchunk + (REV ? a.nchunk - 1 : 0)) * a.groups + g;
    float4* m = a.maps + first * (kSsmVec * 32) + k * 32 + lane;
    const float4* sums = reinterpret_cast<const float4*>(a.sums + first * W::CW + cw);
    constexpr int AHEAD = 24;
    for (int q = 0; q < a.nchunk; q += AHEAD) {
        float4 v[AHEAD], s[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (q + u < a.nchunk - 1) {
                v[u] = __ldcg(m + (q + u) * step * (kSsmVec * 32));
                s[u] = __ldcg(sums + (q + u) * step * (W::CW / 4));
            }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (q + u >= a.nchunk) break;
            m[(q + u) * step * (kSsmVec * 32)] = make_float4(h[0], h[1], h[2], h[3]);
            if (q + u == a.nchunk - 1) break;
            const float e[4] = {v[u].x, v[u].y, v[u].z, v[u].w}, d[4] = {s[u].x, s[u].y, s[u].z, s[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = isinf(d[j]) ? e[j] : fmaf(ex2_approx(A[j] * d[j]), h[j], e[j]);
        }
    }
}

template <int LN, bool KEEP>
__global__ void __launch_bounds__(kSsmWarps * 32, kSsmCtas) ssm_replay_kernel(const SsmArgs a) {
    using W = SsmWarp<LN>;
    constexpr int T = FwdTile<LN, true>::T, IT = (T + W::RPI - 1) / W::RPI;
    extern __shared__ __align__(16) uint8_t buf[];
    pdl_wait();
    const int lane = threadIdx.x & 31, ln = lane % LN, lc = lane / LN;
    const SsmPlace p = place(a, a.nchunk, 0);
    if (!p.on) return;
    FwdTile<LN, true>& s = reinterpret_cast<FwdTile<LN, true>*>(buf)[p.warp];
    const int c0 = p.group * W::CW, ch = c0 + lc * kSsmCh;
    SsmStates A, h;
    load_rates(a.a_log, a.rate_quads, ch, ln * kSsmSt, a.D, a.N, A);
    if (a.nchunk > 1)
        load_tile_state(a.maps + (((long long)p.b * a.nchunk + p.chunk) * a.groups + p.group) * (kSsmVec * 32), lane, h);
    else
        load_state(a.h0, a.quads, p.b, ch, ln * kSsmSt, a.D, a.N, h);
    const int c8 = lane % W::RL * 8, r0 = lane / W::RL;
    const bool on = c0 + c8 < a.D;
    f2x skip[4];
    load_pairs(a.d_skip == nullptr ? nullptr : a.d_skip + c0 + c8, on, skip);
    const int begin = p.chunk * a.chunk, end = min(a.L, begin + a.chunk);
    const int slots = (a.L + kSsmKeep - 1) / kSsmKeep;
    stage_bias<LN>(a.delta_bias, c0, a.D, s.bias, lane);
    FwdRows rows = rows_from(a, p.b, begin, c0);
    ask_tile<LN, true>(a, rows, min(T, end - begin), a.D - c0, s, 0, lane);
    for (int t0 = begin, q = 0; t0 < end; t0 += T, q ^= 1) {
        const int nt = min(T, end - t0);
        const uint32_t starts = start_bits(a.reset, (long long)p.b * a.L + t0, nt, lane);
        copies_wait();
        __syncwarp();
        stage_tile<LN, true>(a, p.b, c0, t0, nt, s, q, lane);
        __syncwarp();
        if (t0 + T < end) ask_tile<LN, true>(a, rows, min(T, end - t0 - T), a.D - c0, s, q ^ 1, lane);
        if (KEEP && t0 % kSsmKeep == 0)
            store_tile_state(a.keep + (((long long)p.b * slots + t0 / kSsmKeep) * a.groups + p.group) * (kSsmVec * 32), lane, h);
        // A token's sums take the place of its dt: every lane of a channel has read that before it takes part in the sum.
        if (starts == 0u) {
#pragma unroll
            for (int t = 0; t < T; ++t) {
                f2x y2[2], dt[2];
                float y[kSsmCh];
                advance<LN, true>(s, t, lc, ln, A, h, y2, dt);
                sum_states<LN>(y2, y, lane);
                put_channels<LN>(s.dt[t], y, lc, ln);
            }
        } else {
#pragma unroll 1
            for (int t = 0; t < T; ++t) {
                if ((starts >> t) & 1u) clear_states(h);
                f2x y2[2], dt[2];
                float y[kSsmCh];
                advance<LN, true>(s, t, lc, ln, A, h, y2, dt);
                sum_states<LN>(y2, y, lane);
                put_channels<LN>(s.dt[t], y, lc, ln);
            }
        }
        __syncwarp();
        if (on) {
            uint16_t* py = a.y + ((long long)p.b * a.L + t0) * a.D + c0 + c8;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * W::RPI;
                if (r >= nt) break;
                f2x y[4], x[4];
                read_pairs(&s.dt[r][c8], y);
                unpack_pairs(*reinterpret_cast<const uint4*>(&s.x[q][r][c8]), x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (a.d_skip != nullptr) y[e] = fma2(skip[e], x[e], y[e]);
                if (a.gate.p != nullptr) {
                    f2x z[4];
                    unpack_pairs(*reinterpret_cast<const uint4*>(&s.gate[q][r][c8]), z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float z0, z1;
                        up2(z[e], z0, z1);
                        y[e] = mul2(y[e], mul2(z[e], pk2(ssm_sigmoid(z0), ssm_sigmoid(z1))));
                    }
                }
                *reinterpret_cast<uint4*>(py + (long long)r * a.D) =
                    make_uint4(x2bf(y[0]), x2bf(y[1]), x2bf(y[2]), x2bf(y[3]));
            }
        }
    }
    pdl_trigger();   // not before: see ssm_maps_kernel
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;
    if (p.chunk == a.nchunk - 1) store_state(a.hT, a.quads, p.b, ch, ln * kSsmSt, a.D, a.N, h);
}

// One token of each of B sequences: LQ lanes share a channel, four states each
// (16 bytes of the state row), and go through the batch.  Bound by the state, read
// and written once in FP32 (256 sequences of 2048 channels and 16 states: 67 MB).
// While it computes a sequence a thread asks for the next one's inputs (1024 sequences of
// 4096 channels and 64 states, 2.1 GB: 440 us, 4.9 TB/s of a copy's 6.8, else 559; the 67
// MB above, which stay in L2 between calls, 15 us, else 17).  Asking further ahead costs
// warps and is slower (two sequences ahead 19 us and 491).
constexpr int kStepThreads = 256, kStepCtas = 4;
// What a thread reads of a sequence; b and c as BF16 pairs.
struct StepInputs {
    float h[4];
    uint32_t b[2], c[2];
    uint16_t x, delta, z;
    uint8_t start;
};
// VEC: the state, b and c four at a time.
template <bool VEC>
__device__ __forceinline__ void load_step(const SsmArgs& a, const float* state, long long b, int c, int n0, bool on,
                                          const bool (&live)[4], StepInputs& q) {
    const float* ps = state + (b * a.D + c) * a.N + n0;
    const uint16_t *pb = a.b.p + b * a.b.sb + n0, *pc = a.c.p + b * a.c.sb + n0;
    q = {};
    if (VEC) {
        if (live[0]) {
            const float4 v = *reinterpret_cast<const float4*>(ps);
            const uint2 vb = __ldg(reinterpret_cast<const uint2*>(pb)), vc = __ldg(reinterpret_cast<const uint2*>(pc));
            q.h[0] = v.x;
            q.h[1] = v.y;
            q.h[2] = v.z;
            q.h[3] = v.w;
            q.b[0] = vb.x;
            q.b[1] = vb.y;
            q.c[0] = vc.x;
            q.c[1] = vc.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (live[e]) {
                q.h[e] = ps[e];
                q.b[e / 2] |= (uint32_t)__ldg(pb + e) << (e % 2 * 16);
                q.c[e / 2] |= (uint32_t)__ldg(pc + e) << (e % 2 * 16);
            }
    }
    if (on) {
        q.x = __ldg(a.x.p + b * a.x.sb + c);
        q.delta = __ldg(a.delta.p + b * a.delta.sb + c);
        if (a.gate.p != nullptr) q.z = __ldg(a.gate.p + b * a.gate.sb + c);
    }
    if (a.reset != nullptr) q.start = __ldg(a.reset + b);
}
template <int LQ, bool VEC>
__global__ void __launch_bounds__(kStepThreads, kStepCtas) ssm_step_kernel(const SsmArgs a, float* __restrict__ state) {
    pdl_trigger();
    pdl_wait();
    const int n0 = threadIdx.x % LQ * 4, c = blockIdx.x * (kStepThreads / LQ) + threadIdx.x / LQ;
    const bool on = c < a.D;
    float A[4];
    bool live[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        live[e] = on && n0 + e < a.N;
        A[e] = live[e] ? ssm_rate(__ldg(a.a_log + (long long)c * a.N + n0 + e)) : 0.f;
    }
    const float bias = on && a.delta_bias != nullptr ? __ldg(a.delta_bias + c) : 0.f;
    const float skip = on && a.d_skip != nullptr ? __ldg(a.d_skip + c) : 0.f;
    StepInputs next = {};
    if (blockIdx.y < a.B) load_step<VEC>(a, state, blockIdx.y, c, n0, on, live, next);
    for (long long b = blockIdx.y; b < a.B; b += gridDim.y) {
        StepInputs q = next;
        if (b + gridDim.y < a.B) load_step<VEC>(a, state, b + gridDim.y, c, n0, on, live, next);
        float bb[4], cc[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            up2(bf2x(q.b[e]), bb[2 * e], bb[2 * e + 1]);
            up2(bf2x(q.c[e]), cc[2 * e], cc[2 * e + 1]);
        }
        const float x = bf_up(q.x), z = bf_up(q.z);
        float dt, unused;
        up2(softplus2(dup2(bf_up(q.delta) + bias)), dt, unused);
        const float k = dt * x;
        float y = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q.h[e] = q.start != 0 ? k * bb[e] : fmaf(ex2_approx(fmaf(A[e], dt, kEx2Low)), q.h[e], k * bb[e]);
            y = fmaf(q.h[e], cc[e], y);
        }
        float* ps = state + (b * a.D + c) * a.N + n0;
        if (VEC) {
            if (live[0]) *reinterpret_cast<float4*>(ps) = make_float4(q.h[0], q.h[1], q.h[2], q.h[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (live[e]) ps[e] = q.h[e];
        }
#pragma unroll
        for (int m = LQ / 2; m >= 1; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (on && n0 == 0) {
            y = fmaf(skip, x, y);
            if (a.gate.p != nullptr) y *= z * ssm_sigmoid(z);
            a.y[b * a.D + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        }
    }
}

template <int LN>
cudaError_t fwd_as(const SsmArgs& a, int what, cudaStream_t s, bool pdl) {
    const SsmSplit w = ssm_split(a.D, a.N);
    const dim3 block((unsigned)w.warps * 32);
    if (what == 0) {
        const size_t smem = w.warps * sizeof(FwdTile<LN, false>), most = kSsmWarps * sizeof(FwdTile<LN, false>);
        static std::atomic<bool> allowed[64];
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_maps_kernel<LN>), most, allowed);
        if (e != cudaSuccess) return e;
        return launch_ex(ssm_maps_kernel<LN>, dim3((unsigned)((long long)a.B * (a.nchunk - 1) * a.ngq)), block, smem, s, pdl, a);
    }
    if (what == 1)
        return launch_ex(ssm_prefix_kernel<LN, false>, dim3((unsigned)((long long)a.B * a.groups * (kSsmVec * 32 / kPrefixThreads))), dim3(kPrefixThreads), 0, s, pdl, a);
    if (what == 2)
        return launch_ex(ssm_prefix_kernel<LN, true>, dim3((unsigned)((long long)a.B * a.groups * (kSsmVec * 32 / kPrefixThreads))), dim3(kPrefixThreads), 0, s, pdl, a);
    const size_t smem = w.warps * sizeof(FwdTile<LN, true>), most = kSsmWarps * sizeof(FwdTile<LN, true>);
    const dim3 grid((unsigned)((long long)a.B * a.nchunk * a.ngq));
    if (a.keep != nullptr) {
        static std::atomic<bool> allowed[64];
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_replay_kernel<LN, true>), most, allowed);
        if (e != cudaSuccess) return e;
        return launch_ex(ssm_replay_kernel<LN, true>, grid, block, smem, s, pdl, a);
    }
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(ssm_replay_kernel<LN, false>), most, allowed);
    if (e != cudaSuccess) return e;
    return launch_ex(ssm_replay_kernel<LN, false>, grid, block, smem, s, pdl, a);
}
cudaError_t fwd(const SsmArgs& a, int what, cudaStream_t s, bool pdl) {
    switch (ssm_split(a.D, a.N).lanes) {
        case 1: return fwd_as<1>(a, what, s, pdl);
        case 2: return fwd_as<2>(a, what, s, pdl);
        case 4: return fwd_as<4>(a, what, s, pdl);
        default: return fwd_as<8>(a, what, s, pdl);
    }
}

template <int LQ>
cudaError_t step_as(const SsmArgs& a, float* state, cudaStream_t s, bool pdl) {
    const int across = (a.D + kStepThreads / LQ - 1) / (kStepThreads / LQ);
    // what the SMs hold at once (or, where that leaves many places empty, a few times over), the batch in equal turns
    const int places = kStepCtas * kSsmSms;
    int most = 1;
    double best = 0.0;
    for (int waves = 1; waves <= 4; ++waves) {
        const int n = std::max(1, std::min(65535, places * waves / across));
        const double used = (double)across * n / ((double)places * waves) - 0.1 * (waves - 1);
        if (used > best) {
            best = used;
            most = n;
        }
    }
    const int turns = (a.B + most - 1) / most;
    const dim3 grid((unsigned)across, (unsigned)((a.B + turns - 1) / turns));
    if (a.state_words) return launch_ex(ssm_step_kernel<LQ, true>, grid, dim3(kStepThreads), 0, s, pdl, a, state);
    return launch_ex(ssm_step_kernel<LQ, false>, grid, dim3(kStepThreads), 0, s, pdl, a, state);
}

}  // namespace

SsmSplit ssm_split(int D, int N) {
    SsmSplit w;
    w.lanes = N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8;
    w.channels = 32 / w.lanes * kSsmCh;
    w.groups = (D + w.channels - 1) / w.channels;
    w.ctas = (w.groups + kSsmWarps - 1) / kSsmWarps;
    w.warps = (w.groups + w.ctas - 1) / w.ctas;
    return w;
}
// As many chunks as give every SM `ctas` CTAs, of 16 tokens at least; one where
// `fewest` would not fit (the maps cost more than they bring).  Not more than
// sqrt(10 L): a warp alone takes about 0.3 us for a token of its chunk (maps and
// replay), the prefix 0.03 us for a chunk (1 x 32768 x 8 with 16 states: 572 chunks
// 77 us, 286 of them 93, 724 of them 85).
void ssm_chunks(int B, int L, int D, int N, int ctas, int fewest, int* chunk, int* nchunk) {
    const SsmSplit w = ssm_split(D, N);
    const long long most = (long long)kSsmSms * ctas / ((long long)B * w.ctas);
    long long n = std::min<long long>(most, (L + 15) / 16);
    n = std::min<long long>(n, std::max(1LL, (long long)std::sqrt(10.0 * L)));
    if (n < fewest) n = 1;
    *chunk = (int)(((L + n - 1) / n + 7) / 8 * 8);
    *nchunk = (L + *chunk - 1) / *chunk;
}
cudaError_t launch_ssm_maps(const SsmArgs& a, cudaStream_t s, bool pdl) { return fwd(a, 0, s, pdl); }
cudaError_t launch_ssm_prefix(const SsmArgs& a, bool reverse, cudaStream_t s, bool pdl) {
    return fwd(a, reverse ? 2 : 1, s, pdl);
}
cudaError_t launch_ssm_replay(const SsmArgs& a, cudaStream_t s, bool pdl) { return fwd(a, 3, s, pdl); }
cudaError_t launch_ssm_step(const SsmArgs& a, float* state, cudaStream_t s, bool pdl) {
    if (a.N <= 4) return step_as<1>(a, state, s, pdl);
    if (a.N <= 8) return step_as<2>(a, state, s, pdl);
    if (a.N <= 16) return step_as<4>(a, state, s, pdl);
    if (a.N <= 32) return step_as<8>(a, state, s, pdl);
    return step_as<16>(a, state, s, pdl);
}

}  // namespace lrs

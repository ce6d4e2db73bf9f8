// Short causal convolution of every channel with its own W = 2, 3 or 4 taps, a
// bias and SiLU, over sequences that may be packed into a row and may go on from
// carried inputs; its backward; and one token of it.
//
//   pre_t = bias + sum_j w_j x_(t-j) over the taps that no sequence start cuts
//           (a start at t - j + 1 .. t cuts tap j), inputs before the row from `state`
//   y_t   = SiLU(pre_t), or pre_t
//   dpre  = dy SiLU'(pre),  dx_t = sum_j w_j dpre_(t+j),  dw_j = sum_t dpre_t x_(t-j)
//
// 4 bytes a value forward, 6 backward.  A thread walks along time through a run of
// tokens of 4 channels, the last W inputs in registers, and asks for 8 rows at a
// time, the next 8 while it computes these.  The backward forms pre again (x is read
// anyway, pre is not kept) and keeps the sums of the dx of the last W tokens.  A run's
// first W - 1 rows, and backward the W - 1 after it, are gone through twice.
//   16 x 4096 x 1024, W = 4: forward 51 us, 5.2 TB/s (0.77 of a copy's measured 6.8);
//   backward 104 us, 3.9 TB/s: about 25 instructions a value, by 8 warps an SM.
//   4 x 4096 x 1024: 17 and 30 us, of which the launches' start and end are 3 us each.
// With 2 channels a thread (twice the warps) 4 x 4096 x 1024 took 23 and 39 us.
#include <algorithm>
#include <type_traits>

#include "ssm.cuh"

namespace lrs {

namespace {

constexpr int kConvStep = 8;      // rows that a thread asks for at a time
constexpr int kConvWarps = 4;     // runs of a CTA
constexpr int P = 2;              // pairs of channels, a thread
constexpr int kConvRun = 80;       // tokens of a run at most
constexpr int kConvSms = 152;
// Resident per SM, by registers.  Backward with 3 at W = 4 (spills) 4 x 4096 x 1024 takes 32 us, 2 x 32768 x 1024 with
// 2 at W = 3 95 us, so 30 and 82.
constexpr int kConvFwdCtas = 5;
constexpr int conv_bwd_ctas(int W) { return W == 4 ? 2 : 3; }

// A launch's CTAs: runs of a batch row by spans of channels.
long long conv_tiles(int B, int L, int run) { return (long long)B * (((long long)L + run * kConvWarps - 1) / (run * kConvWarps)); }
long long conv_spans(int D) { return (D + 64 * P - 1) / (64 * P); }
// A run's tokens: those that end soonest, by the rounds that the SMs take with `ctas` CTAs each and a run's own cost, about
// a step (1 x 8192 x 2560: 72 tokens, one round of 4 CTAs an SM, 39 us backward, 64 tokens 49; 16 x 4096 x 1024: 64 tokens 51 us forward, 80
// tokens 55).  kConvRun at most: what the words of Starts cover.
int conv_run(int B, int L, int D, int ctas) {
    const long long places = (long long)ctas * kConvSms;
    int best = kConvStep;
    long long least = -1;
    for (int run = kConvStep; run <= kConvRun; run += kConvStep) {
        const long long n = conv_tiles(B, L, run) * conv_spans(D);
        const long long cost = (n + places - 1) / places * (run + kConvStep);
        if (least < 0 || cost < least) {
            least = cost;
            best = run;
        }
    }
    return best;
}

// A thread's channels of a row: BF16 words, FP32 pairs.
struct Words {
    uint32_t w[P];
};
__device__ __forceinline__ Words no_words() {
    Words o;
#pragma unroll
    for (int e = 0; e < P; ++e) o.w[e] = 0u;
    return o;
}
__device__ __forceinline__ Words load_words(const uint16_t* p) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
    return {{q.x, q.y}};
}
__device__ __forceinline__ void store_words(uint16_t* p, const Words& o) {
    *reinterpret_cast<uint2*>(p) = make_uint2(o.w[0], o.w[1]);
}
__device__ __forceinline__ void unpack_words(const Words& q, f2x (&v)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = bf2x(q.w[e]);
}
__device__ __forceinline__ void load_vector(const float* p, f2x (&v)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const float2 q = __ldg(reinterpret_cast<const float2*>(p) + e);
        v[e] = pk2(q.x, q.y);
    }
}
__device__ __forceinline__ void clear(f2x (&v)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = 0ull;
}
__device__ __forceinline__ void add_product(f2x (&acc)[P], const f2x (&a)[P], const f2x (&b)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = fma2(a[e], b[e], acc[e]);
}
// A window moves on by a token: v[1 ..] <- v[0 ..].
template <int W>
__device__ __forceinline__ void shift_in(f2x (&v)[W][P]) {
#pragma unroll
    for (int j = W - 1; j > 0; --j)
#pragma unroll
        for (int e = 0; e < P; ++e) v[j][e] = v[j - 1][e];
}
// The starts of a run's tokens and of those around it, as bits of three words: bit 0 is the token 8 before the step that
// the thread is at.  All of the run's are asked for at once (a step's own, asked for with its rows, would be waited for).
struct Starts {
    uint32_t m[3];
};
// (by a whole warp; none outside the row)
__device__ __forceinline__ Starts starts_of(const uint8_t* reset, long long row, int t0, int L, int lane) {
    Starts s = {{0u, 0u, 0u}};
    if (reset == nullptr) return s;
    bool on[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int t = t0 - 8 + 32 * k + lane;
        on[k] = t >= 0 && t < L && __ldg(reset + row + t) != 0;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) s.m[k] = __ballot_sync(0xffffffffu, on[k]);
    return s;
}
// The starts of a step's tokens and the H before, the last token's lowest; moves on by a step.
template <int H>
__device__ __forceinline__ uint32_t next_starts(Starts& s) {
    const uint32_t history = __brev(s.m[0]) >> 16 & ((1u << (kConvStep + H)) - 1u);
#pragma unroll
    for (int k = 0; k < 3; ++k) s.m[k] = __funnelshift_r(s.m[k], k < 2 ? s.m[k < 2 ? k + 1 : 2] : 0u, kConvStep);
    return history;
}
// Whether tap j is inside its sequence: no start at the last j tokens of the history.
__device__ __forceinline__ bool tap_live(uint32_t history, int j) { return (history & ((1u << j) - 1u)) == 0u; }

__device__ __forceinline__ f2x silu2(f2x v) {
    float a, b;
    up2(v, a, b);
    return mul2(v, pk2(ssm_sigmoid(a), ssm_sigmoid(b)));
}

struct ConvPlace {
    int b, c, t0, end;   // batch row, first channel, the run's tokens
    long long tile;      // of the CTA: its runs of one batch row
    bool on;
};
// width: channels of a warp
__device__ __forceinline__ ConvPlace conv_place(const ConvArgs& a, int run, int width) {
    ConvPlace p;
    const int spans = (a.D + width - 1) / width, tiles = (a.L + run * kConvWarps - 1) / (run * kConvWarps);
    p.c = (int)(blockIdx.x % spans) * width + (threadIdx.x & 31) * (width / 32);
    p.tile = blockIdx.x / spans;
    p.b = (int)(p.tile / tiles);
    p.t0 = ((int)(p.tile % tiles) * kConvWarps + (threadIdx.x >> 5)) * run;
    p.end = min(a.L, p.t0 + run);
    p.on = p.c < a.D && p.t0 < a.L;
    return p;
}
// The input at token t of the row (before it: the carried ones).
template <int W>
__device__ __forceinline__ Words conv_input(const ConvArgs& a, int b, int c, int t) {
    if (t >= 0) return load_words(a.x.p + (long long)b * a.x.sb + (long long)t * a.x.st + c);
    if (a.state != nullptr) return load_words(a.state + ((long long)b * (W - 1) + W - 1 + t) * a.D + c);
    return no_words();
}

// bias + the taps that are live; v holds the last W inputs, the newest first.
template <int W, bool CUT>
__device__ __forceinline__ void conv_sum(const f2x (&w)[W][P], const f2x (&bias)[P], const f2x (&v)[W][P], uint32_t history,
                                         f2x (&acc)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        if (CUT && !tap_live(history, j)) break;   // nor any earlier input
        add_product(acc, w[j], v[j]);
    }
}

// kConvStep tokens forward.  PLAIN: all of them there, and no start reaches their
// taps (a group without branches: with a test a token it took twice the instructions).
template <int W, bool SILU, bool PLAIN>
__device__ __forceinline__ void conv_group(const Words (&q)[kConvStep], int n, uint32_t history, const f2x (&w)[W][P],
                                           const f2x (&bias)[P], f2x (&v)[W][P], uint16_t* py, long long ld) {
#pragma unroll
    for (int r = 0; r < kConvStep; ++r) {
        shift_in(v);
        unpack_words(q[r], v[0]);
        if (!PLAIN && r >= n) continue;
        f2x acc[P];
        conv_sum<W, !PLAIN>(w, bias, v, history >> (kConvStep - 1 - r), acc);
        Words o;
#pragma unroll
        for (int e = 0; e < P; ++e) o.w[e] = x2bf(SILU ? silu2(acc[e]) : acc[e]);
        store_words(py + r * ld, o);
    }
}

template <int W, bool SILU>
__global__ void __launch_bounds__(32 * kConvWarps, kConvFwdCtas) causal_conv_fwd_kernel(const ConvArgs a, int run) {
    constexpr int H = W - 1;
    pdl_trigger();
    pdl_wait();
    const ConvPlace p = conv_place(a, run, 64 * P);
    const long long row = (long long)p.b * a.L;
    Starts starts = starts_of(a.reset, row, p.t0, a.L, threadIdx.x & 31);
    if (!p.on) return;
    f2x w[W][P], bias[P], v[W][P];
    clear(bias);
#pragma unroll
    for (int j = 0; j < W; ++j) load_vector(a.w + (long long)j * a.D + p.c, w[j]);
    if (a.bias != nullptr) load_vector(a.bias + p.c, bias);
#pragma unroll
    for (int j = 0; j < H; ++j) unpack_words(conv_input<W>(a, p.b, p.c, p.t0 - 1 - j), v[j]);
    const uint16_t* px = a.x.p + (long long)p.b * a.x.sb + (long long)p.t0 * a.x.st + p.c;
    uint16_t* py = a.y + (row + p.t0) * a.D + p.c;
    Words next[kConvStep];
#pragma unroll
    for (int r = 0; r < kConvStep; ++r) next[r] = r < p.end - p.t0 ? load_words(px + r * a.x.st) : no_words();
    for (int t = p.t0; t < p.end; t += kConvStep, py += (long long)kConvStep * a.D) {
        const int n = p.end - t;
        Words q[kConvStep];
        px += kConvStep * a.x.st;
#pragma unroll
        for (int r = 0; r < kConvStep; ++r) {
            q[r] = next[r];
            next[r] = r + kConvStep < n ? load_words(px + r * a.x.st) : no_words();
        }
        const uint32_t history = next_starts<H>(starts);
        if (n >= kConvStep && history == 0u)
            conv_group<W, SILU, true>(q, n, 0u, w, bias, v, py, a.D);
        else
            conv_group<W, SILU, false>(q, n, history, w, bias, v, py, a.D);
    }
    // the row's last inputs, as far as they belong to its last sequence
    if (a.state_out != nullptr && p.end == a.L) {
        uint32_t history = 0u;
        if (a.reset != nullptr)
#pragma unroll
            for (int k = 0; k < H; ++k)
                if (a.L > k && __ldg(a.reset + row + a.L - 1 - k) != 0) history |= 1u << k;
#pragma unroll
        for (int k = 0; k < H; ++k)   // the input k tokens before the last
            store_words(a.state_out + ((long long)p.b * H + H - 1 - k) * a.D + p.c,
                        tap_live(history, k) ? conv_input<W>(a, p.b, p.c, a.L - 1 - k) : no_words());
    }
}

// One token of each of B sequences; the carried inputs move on in place.
template <int W, bool SILU>
__global__ void __launch_bounds__(128) causal_conv_step_kernel(const ConvArgs a) {
    constexpr int H = W - 1;
    pdl_trigger();
    pdl_wait();
    const int nv = a.D / 8;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)a.B * nv) return;
    const long long b = i / nv;
    const int c = (int)(i - b * nv) * 8;
    const bool start = a.reset != nullptr && __ldg(a.reset + b) != 0;
    uint4 rows[W];
#pragma unroll
    for (int k = 0; k < H; ++k)
        rows[k] = start ? make_uint4(0u, 0u, 0u, 0u)
                        : *reinterpret_cast<const uint4*>(a.state_out + (b * H + k) * a.D + c);
    rows[H] = __ldg(reinterpret_cast<const uint4*>(a.x.p + b * a.x.sb + c));
    f2x acc[4];
    load_pairs(a.bias == nullptr ? nullptr : a.bias + c, true, acc);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        f2x w[4], v[4];
        load_pairs(a.w + (long long)j * a.D + c, true, w);
        unpack_pairs(rows[H - j], v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j == 0 || !start) acc[e] = fma2(w[e], v[e], acc[e]);
    }
    if (SILU)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = silu2(acc[e]);
    *reinterpret_cast<uint4*>(a.y + b * a.D + c) = make_uint4(x2bf(acc[0]), x2bf(acc[1]), x2bf(acc[2]), x2bf(acc[3]));
#pragma unroll
    for (int k = 0; k < H; ++k) *reinterpret_cast<uint4*>(a.state_out + (b * H + k) * a.D + c) = rows[k + 1];
}

__device__ __forceinline__ void put_channels_of(void* p, long long at, bool f32, const f2x (&v)[P]) {
    if (!f32) {
        Words o;
#pragma unroll
        for (int e = 0; e < P; ++e) o.w[e] = x2bf(v[e]);
        store_words(static_cast<uint16_t*>(p) + at, o);
        return;
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
        float2 o;
        up2(v[e], o.x, o.y);
        reinterpret_cast<float2*>(static_cast<float*>(p) + at)[e] = o;
    }
}

// The gradients that a thread adds up along its run, and the sums of dx of the last W tokens.
template <int W>
struct ConvSums {
    f2x dw[W][P], db[P], dx[W][P];
};
// One token backward: d becomes dpre; dx[H - j] of the token j earlier, and the
// weights' sums (in: the token is the run's own).
template <int W, bool SILU, bool CUT>
__device__ __forceinline__ void conv_token_back(const f2x (&w)[W][P], const f2x (&bias)[P], const f2x (&v)[W][P], uint32_t history,
                                                bool in, f2x (&d)[P], ConvSums<W>& s) {
    if (SILU) {
        f2x pre[P];
        conv_sum<W, CUT>(w, bias, v, history, pre);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            float p0, p1;
            up2(pre[e], p0, p1);
            const f2x g = pk2(ssm_sigmoid(p0), ssm_sigmoid(p1)), one = dup2(1.f);
            d[e] = mul2(d[e], mul2(g, fma2(pre[e], sub2(one, g), one)));
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        if (CUT && !tap_live(history, j)) break;
        add_product(s.dx[W - 1 - j], w[j], d);
        if (in) add_product(s.dw[j], d, v[j]);
    }
    if (in)
#pragma unroll
        for (int e = 0; e < P; ++e) s.db[e] = add2(s.db[e], d[e]);
}
// kConvStep tokens backward, of which n are there and `own` the run's own; the first is token `from` of the run.
// PLAIN: all of both, and no start reaches their taps.
template <int W, bool SILU, bool PLAIN>
__device__ __forceinline__ void conv_group_back(const ConvBwdArgs& g, const ConvPlace& p, const Words (&q)[kConvStep],
                                                const Words (&qd)[kConvStep], int n, int own, int from, uint32_t history,
                                                const f2x (&w)[W][P], const f2x (&bias)[P], f2x (&v)[W][P], ConvSums<W>& s) {
    constexpr int H = W - 1;
    const long long at = (long long)p.b * g.dx.sb + (long long)(p.t0 + from - H) * g.dx.st + p.c;
#pragma unroll
    for (int r = 0; r < kConvStep; ++r) {
        if (!PLAIN && r >= own + H) break;
        shift_in(v);
        unpack_words(q[r], v[0]);
        if (PLAIN || r < n) {
            f2x d[P];
            unpack_words(qd[r], d);
            conv_token_back<W, SILU, !PLAIN>(w, bias, v, history >> (kConvStep - 1 - r), PLAIN || r < own, d, s);
        }
        // dx[0] is whole now: the token H earlier.  Before the run it is another thread's, before the row an
        // input carried in.
        if (r >= H || from > 0)
            put_channels_of(g.dx.p, at + r * g.dx.st, g.f32, s.dx[0]);
        else if (p.t0 == 0 && g.dstate != nullptr)
            put_channels_of(g.dstate, ((long long)p.b * H + r) * g.f.D + p.c, g.f32, s.dx[0]);
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) s.dx[j][e] = s.dx[j + 1][e];
        clear(s.dx[H]);
    }
}

template <int W, bool SILU>
__global__ void __launch_bounds__(32 * kConvWarps, conv_bwd_ctas(W)) causal_conv_bwd_kernel(const ConvBwdArgs g, int run) {
    constexpr int H = W - 1;
    __shared__ f2x acc[kConvWarps][W + 1][32][P];
    pdl_trigger();
    pdl_wait();
    const ConvArgs& a = g.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const ConvPlace p = conv_place(a, run, 64 * P);
    const long long row = (long long)p.b * a.L;
    Starts starts = starts_of(a.reset, row, p.t0, a.L, lane);
    ConvSums<W> s;
    clear(s.db);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        clear(s.dw[j]);
        clear(s.dx[j]);
    }
    if (p.on) {
        f2x w[W][P], bias[P], v[W][P];
        clear(bias);
        clear(v[H]);
#pragma unroll
        for (int j = 0; j < W; ++j) load_vector(a.w + (long long)j * a.D + p.c, w[j]);
        if (a.bias != nullptr) load_vector(a.bias + p.c, bias);
#pragma unroll
        for (int j = 0; j < H; ++j) unpack_words(conv_input<W>(a, p.b, p.c, p.t0 - 1 - j), v[j]);
        const uint16_t* px = a.x.p + (long long)p.b * a.x.sb + (long long)p.t0 * a.x.st + p.c;
        const uint16_t* py = g.dy + (row + p.t0) * a.D + p.c;
        // the run's tokens, then the H after it, whose taps reach into it
        Words nq[kConvStep], nqd[kConvStep];
        const int total = min(a.L, p.end + H) - p.t0;
#pragma unroll
        for (int r = 0; r < kConvStep; ++r) {
            nq[r] = nqd[r] = no_words();
            if (r < total) {
                nq[r] = load_words(px + r * a.x.st);
                nqd[r] = load_words(py + (long long)r * a.D);
            }
        }
        for (int t = p.t0; t < p.end + H; t += kConvStep) {
            Words q[kConvStep], qd[kConvStep];
            const int n = min(a.L, p.end + H) - t, own = p.end - t;   // (may be none)
            px += kConvStep * a.x.st;
            py += (long long)kConvStep * a.D;
#pragma unroll
            for (int r = 0; r < kConvStep; ++r) {
                q[r] = nq[r];
                qd[r] = nqd[r];
                nq[r] = nqd[r] = no_words();
                if (r + kConvStep < n) {
                    nq[r] = load_words(px + r * a.x.st);
                    nqd[r] = load_words(py + (long long)r * a.D);
                }
            }
            const uint32_t history = next_starts<H>(starts);
            if (own >= kConvStep && history == 0u)
                conv_group_back<W, SILU, true>(g, p, q, qd, n, own, t - p.t0, 0u, w, bias, v, s);
            else
                conv_group_back<W, SILU, false>(g, p, q, qd, n, own, t - p.t0, history, w, bias, v, s);
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < P; ++e) acc[warp][j][lane][e] = j < W ? s.dw[j < W ? j : 0][e] : s.db[e];
    __syncthreads();
    const int width = 64 * P, spans = (a.D + width - 1) / width;
    for (int i = threadIdx.x; i < (W + 1) * 32 * P; i += 32 * kConvWarps) {
        const int j = i / (32 * P), l = i % (32 * P), c = (int)(blockIdx.x % spans) * width + l * 2;
        if (c >= a.D) continue;
        f2x sum = acc[0][j][l / P][l % P];
#pragma unroll
        for (int k = 1; k < kConvWarps; ++k) sum = add2(sum, acc[k][j][l / P][l % P]);
        float2 o;
        up2(sum, o.x, o.y);
        *reinterpret_cast<float2*>(g.part + (p.tile * (W + 1) + j) * a.D + c) = o;
    }
}

// The parts of dw and dbias joined: 32 columns a CTA, warp k the parts k, k + 32, ...
__global__ void __launch_bounds__(1024) causal_conv_sum_kernel(const ConvBwdArgs g) {
    __shared__ float acc[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, W = g.f.W, D = g.f.D;
    if (blockIdx.x == 0 && threadIdx.x == 0) *g.status = 0u;
    const long long cols = (long long)(W + 1) * D, c = (long long)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int i = k; i < g.parts; i += 32) s += __ldcg(g.part + i * cols + c);
    }
    acc[k][lane] = s;
    __syncthreads();
    if (k != 0 || c >= cols) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += acc[i][lane];
    if (c < (long long)W * D)
        g.dw[c] = s;
    else if (g.dbias != nullptr)
        g.dbias[c - (long long)W * D] = s;
}

template <typename F>
cudaError_t by_width(int W, int silu, F&& f) {
    using std::integral_constant;
    if (silu) {
        if (W == 2) return f(integral_constant<int, 2>(), std::true_type());
        if (W == 3) return f(integral_constant<int, 3>(), std::true_type());
        return f(integral_constant<int, 4>(), std::true_type());
    }
    if (W == 2) return f(integral_constant<int, 2>(), std::false_type());
    if (W == 3) return f(integral_constant<int, 3>(), std::false_type());
    return f(integral_constant<int, 4>(), std::false_type());
}

}  // namespace

int conv_bwd_parts(int B, int L, int D, int W) { return (int)conv_tiles(B, L, conv_run(B, L, D, conv_bwd_ctas(W))); }

cudaError_t launch_causal_conv(const ConvArgs& a, cudaStream_t s, bool pdl) {
    const int run = conv_run(a.B, a.L, a.D, kConvFwdCtas);
    const dim3 grid((unsigned)(conv_tiles(a.B, a.L, run) * conv_spans(a.D)));
    return by_width(a.W, a.silu, [&](auto w, auto silu) {
        return launch_ex(causal_conv_fwd_kernel<decltype(w)::value, decltype(silu)::value>, grid, dim3(32 * kConvWarps), 0, s,
                         pdl, a, run);
    });
}
cudaError_t launch_causal_conv_step(const ConvArgs& a, cudaStream_t s, bool pdl) {
    const dim3 grid((unsigned)(((long long)a.B * (a.D / 8) + 127) / 128));
    return by_width(a.W, a.silu, [&](auto w, auto silu) {
        return launch_ex(causal_conv_step_kernel<decltype(w)::value, decltype(silu)::value>, grid, dim3(128), 0, s, pdl, a);
    });
}
cudaError_t launch_causal_conv_bwd(const ConvBwdArgs& g, cudaStream_t s, bool pdl) {
    const dim3 grid((unsigned)((long long)g.parts * ((g.f.D + 64 * P - 1) / (64 * P))));
    const int run = conv_run(g.f.B, g.f.L, g.f.D, conv_bwd_ctas(g.f.W));
    return by_width(g.f.W, g.f.silu, [&](auto w, auto silu) {
        return launch_ex(causal_conv_bwd_kernel<decltype(w)::value, decltype(silu)::value>, grid, dim3(32 * kConvWarps), 0, s,
                         pdl, g, run);
    });
}
cudaError_t launch_causal_conv_sum(const ConvBwdArgs& g, cudaStream_t s, bool pdl) {
    const long long cols = (long long)(g.f.W + 1) * g.f.D;
    return launch_ex(causal_conv_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s, pdl, g);
}

}  // namespace lrs

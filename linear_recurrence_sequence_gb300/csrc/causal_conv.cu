// Short causal convolution of every channel with its own W = 2, 3 or 4 taps, a
// bias and SiLU, over sequences that may be packed into a row and may go on from
// carried inputs; its backward; and one token of it.
//
//   pre_t = bias + sum_j w_j x_(t-j) over the taps that no sequence start cuts
//           (a start at t - j + 1 .. t cuts tap j), inputs before the row from `state`
//   y_t   = SiLU(pre_t), or pre_t
//   dpre  = dy SiLU'(pre),  dx_t = sum_j w_j dpre_(t+j),  dw_j = sum_t dpre_t x_(t-j)
//
// Bound by bandwidth: 4 bytes a value forward, 6 backward.  A thread forms a run
// of tokens of a few channels and asks for all the rows of its window before any
// arithmetic; the warps of a CTA take neighbouring runs, whose overlapping rows
// meet in L1.  The backward forms pre again (x is read anyway, pre is not kept).
#include <algorithm>

#include "ssm.cuh"

namespace lrs {

namespace {

constexpr int kConvFwdRun = 8;    // tokens of a thread, 8 channels
constexpr int kConvBwdRun = 16;   // tokens of a thread, 4 channels
constexpr int kConvWarps = 8;     // runs of a CTA

// Whether tap j of the token at bit i of the window is inside its sequence: no
// start among the bits i - j + 1 .. i.
__device__ __forceinline__ bool tap_live(uint32_t starts, int i, int j) {
    return ((starts >> (i - j + 1)) & ((1u << j) - 1u)) == 0u;
}
// The starts of tokens t .. t + n - 1 of a row (n <= 32) as bits; none outside it.
template <int n>
__device__ __forceinline__ uint32_t window_starts(const uint8_t* reset, long long row, int t, int L) {
    uint32_t st = 0u;
    if (reset != nullptr)
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (t + i >= 0 && t + i < L && __ldg(reset + row + t + i) != 0) st |= 1u << i;
    return st;
}

__device__ __forceinline__ f2x silu2(f2x v) {
    float a, b;
    up2(v, a, b);
    return mul2(v, pk2(ssm_sigmoid(a), ssm_sigmoid(b)));
}

template <int W, bool SILU>
__global__ void __launch_bounds__(32 * kConvWarps) causal_conv_fwd_kernel(const ConvArgs a) {
    constexpr int R = kConvFwdRun, H = W - 1;
    pdl_trigger();
    pdl_wait();
    const int spans = (a.D + 255) / 256, tiles = (a.L + R * kConvWarps - 1) / (R * kConvWarps);
    const int c = (int)(blockIdx.x % spans) * 256 + (threadIdx.x & 31) * 8;
    const long long bt = blockIdx.x / spans;
    const int b = (int)(bt / tiles), t0 = ((int)(bt % tiles) * kConvWarps + (threadIdx.x >> 5)) * R;
    if (c >= a.D || t0 >= a.L) return;
    const uint16_t* px = a.x.p + (long long)b * a.x.sb + c;
    uint4 rows[R + H];   // inputs t0 - H + i
#pragma unroll
    for (int i = 0; i < R + H; ++i) {
        const int t = t0 - H + i;
        rows[i] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= 0 && t < a.L)
            rows[i] = __ldg(reinterpret_cast<const uint4*>(px + (long long)t * a.x.st));
        else if (t < 0 && a.state != nullptr)
            rows[i] = __ldg(reinterpret_cast<const uint4*>(a.state + ((long long)b * H + H + t) * a.D + c));
    }
    const uint32_t st = window_starts<R + H>(a.reset, (long long)b * a.L, t0 - H, a.L);
    f2x w[W][4], bias[4];
#pragma unroll
    for (int j = 0; j < W; ++j) load_pairs(a.w + (long long)j * a.D + c, true, w[j]);
    load_pairs(a.bias == nullptr ? nullptr : a.bias + c, true, bias);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (t0 + r >= a.L) break;
        f2x acc[4] = {bias[0], bias[1], bias[2], bias[3]};
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (j > 0 && !tap_live(st, r + H, j)) break;   // nor any earlier input
            f2x v[4];
            unpack_pairs(rows[r + H - j], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fma2(w[j][e], v[e], acc[e]);
        }
        if (SILU)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = silu2(acc[e]);
        *reinterpret_cast<uint4*>(a.y + ((long long)b * a.L + t0 + r) * a.D + c) =
            make_uint4(x2bf(acc[0]), x2bf(acc[1]), x2bf(acc[2]), x2bf(acc[3]));
    }
    // the row's last inputs, as far as they belong to its last sequence
    if (a.state_out != nullptr && t0 + R >= a.L) {
#pragma unroll
        for (int i = 0; i < R + H; ++i) {
            const int k = t0 - H + i - (a.L - H);
            if (k < 0 || k >= H) continue;
            const bool live = i == R + H - 1 || (st >> (i + 1)) == 0u;
            *reinterpret_cast<uint4*>(a.state_out + ((long long)b * H + k) * a.D + c) =
                live ? rows[i] : make_uint4(0u, 0u, 0u, 0u);
        }
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

__device__ __forceinline__ void unpack4(const uint2 q, f2x (&v)[2]) {
    v[0] = bf2x(q.x);
    v[1] = bf2x(q.y);
}
__device__ __forceinline__ void put4(void* p, long long at, bool f32, const f2x (&v)[2]) {
    if (f32) {
        float4 o;
        up2(v[0], o.x, o.y);
        up2(v[1], o.z, o.w);
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = o;
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = make_uint2(x2bf(v[0]), x2bf(v[1]));
    }
}

template <int W, bool SILU>
__global__ void __launch_bounds__(32 * kConvWarps) causal_conv_bwd_kernel(const ConvBwdArgs g) {
    constexpr int R = kConvBwdRun, H = W - 1;
    __shared__ float4 acc[kConvWarps][W + 1][32];
    pdl_trigger();
    pdl_wait();
    const ConvArgs& a = g.f;
    const int spans = (a.D + 127) / 128, tiles = (a.L + R * kConvWarps - 1) / (R * kConvWarps);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int)(blockIdx.x % spans) * 128 + lane * 4;
    const long long bt = blockIdx.x / spans;
    const int b = (int)(bt / tiles), t0 = ((int)(bt % tiles) * kConvWarps + warp) * R;
    f2x dw[W][2], db[2] = {0ull, 0ull};
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][0] = dw[j][1] = 0ull;
    if (c < a.D && t0 < a.L) {
        const uint16_t* px = a.x.p + (long long)b * a.x.sb + c;
        const uint16_t* py = g.dy + (long long)b * a.L * a.D + c;
        uint2 rows[R + 2 * H], dys[R + H];   // x from t0 - H on, dy from t0 on
#pragma unroll
        for (int i = 0; i < R + 2 * H; ++i) {
            const int t = t0 - H + i;
            rows[i] = make_uint2(0u, 0u);
            // past the run x only serves pre
            if (t >= 0 && t < a.L && (SILU || i < R + H))
                rows[i] = __ldg(reinterpret_cast<const uint2*>(px + (long long)t * a.x.st));
            else if (t < 0 && a.state != nullptr)
                rows[i] = __ldg(reinterpret_cast<const uint2*>(a.state + ((long long)b * H + H + t) * a.D + c));
        }
#pragma unroll
        for (int i = 0; i < R + H; ++i)
            dys[i] = t0 + i < a.L ? __ldg(reinterpret_cast<const uint2*>(py + (long long)(t0 + i) * a.D))
                                  : make_uint2(0u, 0u);
        const uint32_t st = window_starts<R + 2 * H>(a.reset, (long long)b * a.L, t0 - H, a.L);
        f2x w[W][2], bias[2] = {0ull, 0ull};
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.w + (long long)j * a.D + c));
            w[j][0] = pk2(q.x, q.y);
            w[j][1] = pk2(q.z, q.w);
        }
        if (a.bias != nullptr) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.bias + c));
            bias[0] = pk2(q.x, q.y);
            bias[1] = pk2(q.z, q.w);
        }
        // dx of the tokens t0 + r - H .. t0 + r while r runs
        f2x dx[W][2];
#pragma unroll
        for (int j = 0; j < W; ++j) dx[j][0] = dx[j][1] = 0ull;
#pragma unroll
        for (int r = 0; r < R + H; ++r) {
            f2x d[2];
            unpack4(dys[r], d);
            if (SILU) {
                f2x pre[2] = {bias[0], bias[1]};
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    if (j > 0 && !tap_live(st, r + H, j)) break;
                    f2x v[2];
                    unpack4(rows[r + H - j], v);
                    pre[0] = fma2(w[j][0], v[0], pre[0]);
                    pre[1] = fma2(w[j][1], v[1], pre[1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float p0, p1;
                    up2(pre[e], p0, p1);
                    const f2x s = pk2(ssm_sigmoid(p0), ssm_sigmoid(p1)), one = dup2(1.f);
                    d[e] = mul2(d[e], mul2(s, fma2(pre[e], sub2(one, s), one)));
                }
                if (t0 + r >= a.L) d[0] = d[1] = 0ull;
            }
            // tap j reaches token t0 + r - j, which is dx[H - j] of the window
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (j > 0 && !tap_live(st, r + H, j)) break;
                dx[H - j][0] = fma2(w[j][0], d[0], dx[H - j][0]);
                dx[H - j][1] = fma2(w[j][1], d[1], dx[H - j][1]);
                if (r < R) {
                    f2x v[2];
                    unpack4(rows[r + H - j], v);
                    dw[j][0] = fma2(d[0], v[0], dw[j][0]);
                    dw[j][1] = fma2(d[1], v[1], dw[j][1]);
                }
            }
            if (r < R) {
                db[0] = add2(db[0], d[0]);
                db[1] = add2(db[1], d[1]);
            }
            // the window's first token has all its taps: t0 + r - H.  Before the run it is another
            // thread's, before the row an input carried in.
            const int t = t0 + r - H;
            if (r >= H) {
                if (t < a.L) put4(g.dx.p, (long long)b * g.dx.sb + (long long)t * g.dx.st + c, g.f32, dx[0]);
            } else if (t0 == 0 && g.dstate != nullptr) {
                put4(g.dstate, ((long long)b * H + r) * a.D + c, g.f32, dx[0]);
            }
#pragma unroll
            for (int j = 0; j < H; ++j) {
                dx[j][0] = dx[j + 1][0];
                dx[j][1] = dx[j + 1][1];
            }
            dx[H][0] = dx[H][1] = 0ull;
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float4 o;
        up2(j < W ? dw[j < W ? j : 0][0] : db[0], o.x, o.y);
        up2(j < W ? dw[j < W ? j : 0][1] : db[1], o.z, o.w);
        acc[warp][j][lane] = o;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32; i += 32 * kConvWarps) {
        const int j = i / 32, l = i % 32, cc = (int)(blockIdx.x % spans) * 128 + l * 4;
        if (cc >= a.D) continue;
        float4 v = acc[0][j][l];
#pragma unroll
        for (int k = 1; k < kConvWarps; ++k) {
            const float4 q = acc[k][j][l];
            v.x += q.x;
            v.y += q.y;
            v.z += q.z;
            v.w += q.w;
        }
        *reinterpret_cast<float4*>(g.part + (bt * (W + 1) + j) * a.D + cc) = v;
    }
}

// The parts of dw and dbias joined: 32 columns a CTA, warp k the parts k, k + 32, ...
__global__ void __launch_bounds__(1024) causal_conv_sum_kernel(const ConvBwdArgs g) {
    __shared__ float acc[32][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, W = g.f.W, D = g.f.D;
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

int conv_bwd_parts(int B, int L, int D) {
    const int tokens = kConvBwdRun * kConvWarps;
    return B * ((L + tokens - 1) / tokens);
}

cudaError_t launch_causal_conv(const ConvArgs& a, cudaStream_t s, bool pdl) {
    const long long tiles = (a.L + kConvFwdRun * kConvWarps - 1) / (kConvFwdRun * kConvWarps);
    const dim3 grid((unsigned)(a.B * tiles * ((a.D + 255) / 256)));
    return by_width(a.W, a.silu, [&](auto w, auto silu) {
        return launch_ex(causal_conv_fwd_kernel<decltype(w)::value, decltype(silu)::value>, grid, dim3(32 * kConvWarps), 0, s,
                         pdl, a);
    });
}
cudaError_t launch_causal_conv_step(const ConvArgs& a, cudaStream_t s, bool pdl) {
    const dim3 grid((unsigned)(((long long)a.B * (a.D / 8) + 127) / 128));
    return by_width(a.W, a.silu, [&](auto w, auto silu) {
        return launch_ex(causal_conv_step_kernel<decltype(w)::value, decltype(silu)::value>, grid, dim3(128), 0, s, pdl, a);
    });
}
cudaError_t launch_causal_conv_bwd(const ConvBwdArgs& g, cudaStream_t s, bool pdl) {
    const dim3 grid((unsigned)((long long)g.parts * ((g.f.D + 127) / 128)));
    return by_width(g.f.W, g.f.silu, [&](auto w, auto silu) {
        return launch_ex(causal_conv_bwd_kernel<decltype(w)::value, decltype(silu)::value>, grid, dim3(32 * kConvWarps), 0, s,
                         pdl, g);
    });
}
cudaError_t launch_causal_conv_sum(const ConvBwdArgs& g, cudaStream_t s, bool pdl) {
    const long long cols = (long long)(g.f.W + 1) * g.f.D;
    return launch_ex(causal_conv_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s, pdl, g);
}

}  // namespace lrs

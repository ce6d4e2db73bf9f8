// Softmax cross entropy over a large vocabulary without keeping the logits:
// the contractions, on the fifth-generation tensor cores (sm_103a).
//
// With hidden states h [T][D], the head w [V][D] and z = h w^T, forward and
// backward are three contractions around row-wise softmax statistics:
//   NT  z = h w^T        a tile of logits lives in tensor memory only; the
//                        epilogue leaves (max, sum of exponentials) of each
//                        row's 128 columns (forward), or
//                        dz = dloss (e^{z - lse} - [v = target]) (backward),
//                        the latter for one piece of the vocabulary at a time;
//   NN  dh = dz w        A = dz [T][piece] K-major, B = w's rows as K index;
//   TN  dw = dz^T h      both operands MN-major, the tokens as K index;
// the last two in one launch: neither's tile count fills the pairs of SMs
// evenly, and together they do (a pair with one dh tile less than the others
// takes as many more of the shorter dw tiles; 8192 tokens x 32768 entries at
// D 2048: 1171 us, one after the other 1267; 16 tokens at D 1024: 37 and 60).
// Measured (events around each launch): the statistics of 32768 x 32768 at
// D 1024 1.07 ms, 2.06 PFLOP/s; dz of 8192 x 32768 at D 2048 0.58 ms, 1.9; dh and
// dw of it 1.17 ms, 1.9.  Back to back such calls meet the power limit, at about
// 1.7.  Unlike the block's contractions (block_gemm.cu) every extent may be ragged:
// the TMA fills what lies outside a matrix with zeros and clips what is stored
// there; columns past the vocabulary are zeroed in dz.
//
// CTA pairs (cta_group::2) take 256 x 256 tiles: each CTA loads its 128 rows
// of A and half of B's slice, so the pair reads every operand value of its tile
// once and shared memory holds three 128-wide K slices of it.  In each CTA warp 8
// streams the slices by TMA (128-byte swizzle), completing on the even CTA's
// barriers; one thread of the even CTA's warp 9 issues tcgen05.mma (M 256,
// N 256, K 16) for both and frees the slices by commits to both; warps 0-7
// drain the CTA's 128 accumulator rows, of which there are two sets in turn so
// that a tile's epilogue runs under the next tile's MMAs.  Every wait is
// bounded but the pair's allocation of tensor memory, which waits for kernels
// that hold columns on either SM; those end by themselves (their waits are
// bounded), and both CTAs of a cluster are resident together.
#include <algorithm>
#include <atomic>

#include "kernels.cuh"
#include "tmap.cuh"
#include "twosum.cuh"
#include "umma.cuh"

namespace lrs {

namespace {

constexpr int kCeEpiWarps = 8;
constexpr int kCeThreads = 32 * (kCeEpiWarps + 2);
constexpr int kCeProducer = kCeEpiWarps, kCeIssuer = kCeEpiWarps + 1;
constexpr int kCeK = 128;         // K per stage: two 64-wide (128-byte) chunks
constexpr int kCeM = 256;         // rows of a pair's tile: 128 a CTA
constexpr int kCeN = 256;
constexpr int kCeStages = 3;
constexpr uint32_t kCeABytes = 2 * 128 * 128;   // of one CTA: 128 rows of A, 128 of B, two chunks each
constexpr uint32_t kCeBBytes = 2 * 128 * 128;
constexpr uint32_t kCeChunk = 128 * 128;        // a 64-column chunk of 128 rows
constexpr uint32_t kCeStageBytes = kCeABytes + kCeBBytes;
constexpr uint32_t kCeTmemCols = 2 * kCeN;
constexpr uint32_t kCeBox = 32 * 32 * 2;   // a [32 rows][32 columns] BF16 store box (64-byte swizzle)
constexpr uint32_t kCeWideBox = 2 * kCeBox;   // [32][64] (128-byte swizzle)
// Staging of the stores, one box per epilogue warp: BF16 [32 rows][64 columns],
// with parts two of [32][32], taken in turns; FP32 [32][32].
__host__ __device__ constexpr uint32_t ce_stage_warp(int epi) {
    return epi != kCeStats ? kCeWideBox : 0u;
}
constexpr size_t ce_smem(int epi) {
    return (size_t)kCeStages * kCeStageBytes + (size_t)kCeEpiWarps * ce_stage_warp(epi) + 1024;
}

constexpr int kCeFewThreads = 1024;   // per SM, of the kernel for one token (half of it for more)
// The rows of h that it keeps: up to four CTAs of this and their own 1 KB fit an SM.
constexpr size_t kCeFewSmem = 48 * 1024;
// Stages that one accumulator adds up.  The tensor cores' sums lose about 2e-8 of
// their value a step of 16 (they truncate; 8 steps a stage), 6e-5 over 50021
// vocabulary entries in one chain.  Chains add up in registers: those of 8 stages
// keep the loss and lse of any width where D 1024 has them (relative error 5e-7;
// D 4096 in one chain 2e-6), and cost a wide D nothing (8192 tokens x 65536 entries at
// D 2048: 4.49 ms with and without).  FP32 gradients, dh and dw of 2048 x 25088 at
// D 1024 and the error of dw: chains of 2 stages 471 us and 3.7e-7, 3: 391 and 5.1e-7,
// 4: 378 and 6.5e-7, 8: 366 and 1.3e-6.
__host__ __device__ constexpr int ce_chain(int epi) {
    return epi == kCeStats || epi == kCeDz ? 8 : epi == kCeDz3 ? 4 : 3;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(f2_to_bf2(v[0], v[1]), f2_to_bf2(v[2], v[3]), f2_to_bf2(v[4], v[5]), f2_to_bf2(v[6], v[7]));
}

struct CeItem {
    int side;             // contraction (of a.c)
    int mt, nt, s, k0, k1;
    int m0;               // this CTA's first row
};

// Item k of pair `pair`; false where it has no more.
// One contraction (the logits): the pairs take turns, rows fastest inside a
// group of row tiles whose h stays in the L2, so that a tile of w is read by
// the whole group at about the same time.
// Two (dh and dw): dh's items first, in turns; the pairs that get one less
// take `extra` more of dw's.  The tiles of D run fastest, so that those that
// read the same panel of dz run together.
__device__ __forceinline__ bool ce_item(const CeGemmArgs& a, bool grads, int pair, int pairs, int k, int rank, CeItem& it) {
    const CeSide* c = a.c;
    if (!grads) {
        const int i = pair + k * pairs;
        if (i >= c->n_items) return false;
        const int per = a.group * c->n_tiles;
        const int g = i / per, r = i - g * per;
        const int gm = min(a.group, c->m_tiles - g * a.group);
        it.side = 0;
        it.mt = g * a.group + r % gm;
        it.nt = r / gm;
        it.s = 0;
    } else {
        const int n0 = a.c[0].n_items, more = n0 % pairs;
        const int own = n0 / pairs + (pair < more ? 1 : 0);   // dh items of this pair
        int i;
        if (k < own) {
            it.side = 0;
            i = pair + k * pairs;
        } else {
            it.side = 1;
            ++c;
            const int few = pairs - more;                     // pairs with one dh item less
            const int r = k - own;
            if (pair >= more && r < a.extra)
                i = r * few + pair - more;
            else
                i = a.extra * few + (r - (pair >= more ? a.extra : 0)) * pairs + pair;
            if (i >= c->n_items) return false;
        }
        it.nt = i % c->n_tiles;
        const int r = i / c->n_tiles;
        it.mt = r % c->m_tiles;
        it.s = r / c->m_tiles;
    }
    it.m0 = it.mt * kCeM + 128 * rank;
    it.k0 = (int)((long long)c->ksteps * it.s / c->splits);
    it.k1 = (int)((long long)c->ksteps * (it.s + 1) / c->splits);
    return true;
}

// 32 columns of this lane's accumulator row; the warp's lanes meet first (the
// load is one instruction of the whole warp).
__device__ __forceinline__ void ce_columns(uint32_t taddr, float (&v)[2][16]) {
    __syncwarp();
    tmem_ld16x2(taddr, taddr + 16u, v[0], v[1]);
}

// The capped logit, z' = c tanh(z / c); its slope dz'/dz is 1 - (z'/c)^2.
__device__ __forceinline__ float ce_cap(const CeGemmArgs& a, float z) { return a.softcap * tanhf(z * a.inv_softcap); }

// tanh(x) for |x| <= kCeSeries: the first seven terms of its Taylor series (the
// eighth is below 4e-9 of the value there).
constexpr float kCeSeries = 0.4f;
__device__ __forceinline__ float ce_tanh_small(float x) {
    const float x2 = x * x;
    float p = fmaf(x2, 21844.f / 6081075.f, -1382.f / 155925.f);
    p = fmaf(p, x2, 62.f / 2835.f);
    p = fmaf(p, x2, -17.f / 315.f);
    p = fmaf(p, x2, 2.f / 15.f);
    p = fmaf(p, x2, -1.f / 3.f);
    return fmaf(p * x2, x, x);
}
// tanh(x / c) of 32 logits in place (c the cap): the series, 9 operations, where
// |x / c| is small, as logits mostly are, tanhf's about 25, which held the capped
// epilogues back, for the others.  Each element goes by its own size alone, so
// that no result depends on its neighbours in the warp (rows past the matrix among
// them, whose accumulators hold anything); the warp decides together only whether
// any element needs tanhf (2048 tokens x 50021 entries at D 1024, cap 30: statistics
// 145 us with logits of deviation 2.5, 163 by tanhf alone; 200 with deviation 10,
// where most warps form both).
__device__ __forceinline__ void ce_tanh(const CeGemmArgs& a, float (&v)[2][16]) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        v[j / 16][j % 16] *= a.inv_softcap;
        top = fmaxf(top, fabsf(v[j / 16][j % 16]));
    }
    // (a NaN among the logits is not seen by the maximum, and stays one either way)
    if (__any_sync(0xffffffffu, top > kCeSeries)) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float x = v[j / 16][j % 16], far = tanhf(x);
            v[j / 16][j % 16] = fabsf(x) <= kCeSeries ? ce_tanh_small(x) : far;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j / 16][j % 16] = ce_tanh_small(v[j / 16][j % 16]);
    }
}

// The next 32 of this lane's 128 sums; the others move up (a loop over them needs
// registers by constant number).
__device__ __forceinline__ void ce_take(float (&sum)[kCeN / 2], float (&v)[2][16]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j / 16][j % 16] = sum[j];
#pragma unroll
    for (int j = 0; j < kCeN / 2 - 32; ++j) sum[j] = sum[j + 32];
}

// Forward epilogue of one row: (max, sum e^{z - max}) of its 128 columns, read
// from its accumulator or (CHAINS) from `sums`.
// Columns past the vocabulary do not count; the target's logit is kept.
template <bool CAP, bool CHAINS>
__device__ __forceinline__ void ce_epi_stats(const CeGemmArgs& a, const CeItem& it, int row, uint32_t taddr, int half,
                                             float (&sums)[kCeN / 2]) {
    const int t = it.m0 + row;
    const int c0 = half * (kCeN / 2);
    const int v0 = it.nt * kCeN + c0;            // vocabulary index of the first column
    const int nv = min(kCeN / 2, a.c[0].N - v0);      // columns that count (may be <= 0)
    const int M = a.c[0].M;
    const bool ok = t < M;
    long long tgt = -1;
    if (ok) tgt = a.target[t] - v0;
    float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < kCeN / 2; c += 32) {
        float v[2][16];
        if (CHAINS)
            ce_take(sums, v);
        else
            ce_columns(taddr + (uint32_t)(c0 + c), v);
        if (CAP) ce_tanh(a, v);
        if (!ok || c >= nv) continue;
        float z[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = CAP ? a.softcap * v[j / 16][j % 16] : v[j / 16][j % 16];
        if (tgt >= c && tgt < c + 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (tgt == c + j) a.zt[t] = z[j];
        }
        if (nv - c < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j >= nv) z[j] = -INFINITY;
        }
        float m = z[0];
#pragma unroll
        for (int j = 1; j < 32; ++j) m = fmaxf(m, z[j]);
        m = fmaxf(m, mx);
        const float ref = m == -INFINITY ? 0.f : m;   // every logit so far is -inf: e^{-inf - 0} = 0
        const float off = -ref * kLog2e;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) s += ex2_approx(fmaf(z[j], kLog2e, off));
        sum = fmaf(sum, ex2_approx(fmaf(mx, kLog2e, off)), s);
        mx = m;
    }
    if (ok) a.stats[(size_t)(2 * it.nt + half) * M + t] = make_float2(mx, sum);
}

// 32 columns (from c of the tile) of this lane's row as FP32, times `common`:
// staged in the warp's swizzled box and stored, or added, by the TMA, which
// clips rows and columns past the matrix.  (Stores by the threads, a row each,
// touch 32 lines an instruction: 16 tokens x 32768 entries at D 1024, 110 us
// against 67.)
__device__ __forceinline__ void ce_store_f32(const CUtensorMap& map, const CeSide& c0, const CeItem& it, const float* v,
                                             float common, uint8_t* stg, int c, int q4, int lane) {
    if (lane == 0) bulk_wait_read<0>();   // the box is read out
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u)
        *reinterpret_cast<float4*>(stg + (size_t)lane * 128 + 16 * (u ^ (lane & 7))) =
            make_float4(v[4 * u] * common, v[4 * u + 1] * common, v[4 * u + 2] * common, v[4 * u + 3] * common);
    fence_proxy_async();
    __syncwarp();
    const int x = it.nt * kCeN + c, y = it.m0 + 32 * q4;
    if (lane == 0 && x < c0.N && y < c0.M) {
        if (c0.accumulate)
            tma_add_3d(&map, x, y, it.s, stg);
        else
            tma_store_3d(&map, x, y, it.s, stg);
        bulk_commit();
    }
}

// The largest finite |dloss| of the tokens counted (1 where none is above 0): dz
// is rounded to BF16 relative to it, so that equal weights, whatever they are, are
// not rounded at all (one rounding for all tokens would be an error of the whole
// gradient).  A weight that is not finite stays in its own row of dz.  Every CTA's
// epilogue warps find it for themselves, under the first tile's products.
__device__ __forceinline__ float ce_largest_weight(const CeGemmArgs& a, uint32_t* s_weight) {
    uint32_t m = 0u;
    for (int t = threadIdx.x; t < a.T; t += 32 * kCeEpiWarps) {
        const long long tg = __ldg(reinterpret_cast<const long long*>(a.target) + t);
        if (tg >= 0 && tg < a.V) {
            const uint32_t w = __float_as_uint(fabsf(__ldg(a.weights + t)));
            if (w < 0x7f800000u) m = max(m, w);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) atomicMax(s_weight, m);
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kCeEpiWarps) : "memory");
    m = *reinterpret_cast<volatile uint32_t*>(s_weight);
    return m != 0u ? __uint_as_float(m) : 1.f;
}
// w / largest, exactly 1 where they are equal.
__device__ __forceinline__ float ce_ratio(float w, float largest) { return w != 0.f ? __fdiv_rn(w, largest) : 0.f; }

// The rows of h that dw = dz^T h adds up: zeros for tokens that are not counted,
// whatever their rows hold.  Copied by the epilogue warps of the dz kernel, a
// warp a row, under the first tile's products.
__device__ __forceinline__ void ce_rows_of_h(const CeGemmArgs& a, int warp, int lane) {
    const int nv = a.c[0].K / 8;
    for (int t = (int)blockIdx.x * kCeEpiWarps + warp; t < a.T; t += (int)gridDim.x * kCeEpiWarps) {
        const long long tg = a.target[t];
        const bool counted = tg >= 0 && tg < a.V;
        for (int c = lane; c < nv; c += 32) {
            const size_t i = (size_t)t * nv + c;
            a.rows_out[i] = counted ? __ldg(a.rows_in + i) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

// Tensor maps of both contractions: A's parts, B, the result (more: dz's second and third parts).
struct CeMaps {
    CUtensorMap a[kCeParts][2], b[2], s[2], more[kCeParts - 1];
};

// CHAINS: the axis in chains of ce_chain stages, added up in registers.
template <int EPI, bool CAP, bool CHAINS>
__global__ void __launch_bounds__(kCeThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CeMaps tm, const __grid_constant__ CeGemmArgs a) {
    constexpr bool GRADS = EPI == kCeGrads || EPI == kCeGrads3;
    constexpr int S = kCeStages, kChain = ce_chain(EPI);
    extern __shared__ uint8_t ce_raw[];
    // s_full and s_free are used in the even CTA, the others in both
    __shared__ __align__(8) uint64_t s_full[S], s_empty[S], s_acc[2], s_free[2], s_fin;
    __shared__ uint32_t s_tmem, s_weight;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ce_raw) + 1023u) & ~uintptr_t(1023));
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_acc[i], 1);
            mbar_init(&s_free[i], 2 * kCeEpiWarps);
        }
        mbar_init(&s_fin, 1);
        s_abort = 0;
        s_weight = 0u;
    }
    if (warp == kCeIssuer) {
        tmem_alloc2(&s_tmem, kCeTmemCols);
        tmem_fence_before_sync();
    }
    __syncthreads();
    pdl_trigger();   // not before the allocation: see umma.cuh
    pdl_wait();
    // a call's first kernel clears the status word and the rows' ticket (a wait gives up 0.2 s from here at the soonest)
    if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) a.status[0] = a.status[1] = 0u;
    cluster_sync();   // the pair's barriers and tensor memory exist
    tmem_fence_after_sync();
    const uint32_t tmem = s_tmem;
    volatile int* abort_flag = &s_abort;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(a.status, kStatusTimeout);
    };
    const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;   // the same items in both CTAs
    CeItem it;

    if (warp == kCeProducer) {
        if (lane == 0) {
            uint32_t n = 0;
            for (int k = 0; !*abort_flag && ce_item(a, GRADS, pair, pairs, k, rank, it); ++k) {
                const CeSide& c = a.c[it.side];
                const bool tn = GRADS && it.side == 1;
                const CUtensorMap* tb = &tm.b[it.side];
                for (int ks = it.k0; ks < it.k1; ++ks, ++n) {
                    const int slot = (int)(n % S);
                    if (n >= (uint32_t)S && !mbar_wait_bounded(&s_empty[slot], ((n / S) - 1) & 1u)) {
                        fail();
                        break;
                    }
                    if (*abort_flag) break;
                    uint8_t* sa = ring + (size_t)slot * kCeStageBytes;
                    uint8_t* sb = sa + kCeABytes;
                    // the parts of dz follow each other along K
                    const int part = EPI != kCeGrads3 ? 0 : (ks >= c.part_steps) + (ks >= 2 * c.part_steps);
                    const int k0 = kCeK * (ks - part * c.part_steps);
                    const int n0 = it.nt * kCeN + 128 * rank;
                    const CUtensorMap* ta = &tm.a[part][it.side];
                    // both CTAs' bytes are announced by the even one (the odd one's may land first)
                    // rows of A past the matrix (of K-major A past the next eight) are not loaded:
                    // what their accumulator rows hold is not used
                    const uint32_t a_bytes = tn ? kCeABytes : 2 * a.a_chunk;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&s_full[slot],
                                              2 * kCeBBytes + (it.m0 + 128 < c.M ? 2 * a_bytes : a_bytes));
                    const uint32_t bar = cluster_map(&s_full[slot], 0);
                    // each operand as one box of two chunks; where rows are no whole number of chunks (the
                    // second would run into the next row), as two boxes that the matrix's edge cuts
                    const int ax = tn ? it.m0 : k0, ay = tn ? k0 : it.m0;
                    if (it.m0 >= c.M) {
                    } else if (GRADS || a.whole) {
                        tma2_load_3d(sa, ta, 0, ay, ax / 64, bar);
                    } else {
                        tma2_load_2d(sa, ta, ax, ay, bar);
                        tma2_load_2d(sa + a.a_chunk, ta, ax + 64, ay, bar);
                    }
                    const int bx = GRADS ? n0 : k0, by = c.b_row + (GRADS ? k0 : n0);
                    if (a.whole) {
                        tma2_load_3d(sb, tb, 0, by, bx / 64, bar);
                    } else {
                        tma2_load_2d(sb, tb, bx, by, bar);
                        tma2_load_2d(sb + kCeChunk, tb, bx + 64, by, bar);
                    }
                }
            }
            // copies still in flight land (the even CTA's barriers count both CTAs'), and the last slices
            // have been read, before the CTA may exit
            const uint32_t lo = n > (uint32_t)S ? n - S : 0;
            if (rank == 0)
                for (uint32_t j = lo; j < n; ++j) mbar_wait_bounded(&s_full[j % S], (j / S) & 1u);
            for (uint32_t j = lo; j < n; ++j) mbar_wait_bounded(&s_empty[j % S], (j / S) & 1u);
        }
    } else if (warp == kCeIssuer) {
        if (lane == 0 && rank == 0) {
            uint32_t n = 0, use = 0;   // stages consumed, accumulators filled
            bool ok = true;
            for (int k = 0; ok && !*abort_flag && ce_item(a, GRADS, pair, pairs, k, rank, it); ++k) {
                const bool tn = GRADS && it.side == 1;   // A MN-major too
                const uint32_t idesc = umma_idesc_bf16(kCeM, kCeN) | (tn ? (1u << 15) : 0u) | (GRADS ? (1u << 16) : 0u);
                for (int k0 = it.k0; ok && k0 < it.k1; k0 += kChain, ++use) {
                    const int k1 = CHAINS ? min(k0 + kChain, it.k1) : it.k1;
                    const uint32_t buf = use & 1u;
                    // both CTAs' epilogues have drained this accumulator's previous contents
                    if (use >= 2 && !mbar_wait_cluster(&s_free[buf], ((use >> 1) - 1) & 1u)) {
                        fail();
                        ok = false;
                        break;
                    }
                    tmem_fence_after_sync();
                    const uint32_t acc_t = tmem + buf * (uint32_t)kCeN;
                    for (int ks = k0; ks < k1; ++ks, ++n) {
                        const int slot = (int)(n % S);
                        if (!mbar_wait_bounded(&s_full[slot], (n / S) & 1u)) {
                            fail();
                            ok = false;
                            break;
                        }
                        tmem_fence_after_sync();
                        const uint32_t sa = smem_u32(ring + (size_t)slot * kCeStageBytes);
                        const uint32_t sb = sa + kCeABytes;
#pragma unroll
                        for (int kk = 0; kk < kCeK / 16; ++kk) {
                            // K-major: chunk kk / 4, 32 bytes a step; MN-major: 16 rows a step in both chunks
                            const uint32_t at = 32u * (kk % 4), mn = 2048u * kk;
                            const uint64_t da = tn ? umma_desc_sw128_mn(sa + mn, kCeChunk)
                                                   : umma_desc_sw128(sa + (kk < 4 ? at : a.a_chunk + at));
                            const uint64_t db = GRADS ? umma_desc_sw128_mn(sb + mn, kCeChunk)
                                                      : umma_desc_sw128(sb + (kk < 4 ? at : kCeChunk + at));
                            umma2_bf16(acc_t, da, db, idesc, ks > k0 || kk > 0);
                        }
                        umma2_commit(&s_empty[slot]);
                    }
                    if (!ok) break;
                    umma2_commit(&s_acc[buf]);
                    if (!CHAINS) {
                        ++use;
                        break;
                    }
                }
            }
            // every MMA issued by this thread has completed before the columns are released
            umma2_commit_own(&s_fin);
            mbar_wait_bounded(&s_fin, 0);
        }
    } else {
        // epilogue warps: rows 32 (warp % 4) .. + 31 of the CTA's 128, column half warp / 4
        const int q4 = warp & 3, hf = warp >> 2;
        const int row = 32 * q4 + lane;
        uint8_t* stg = ring + (size_t)S * kCeStageBytes + (size_t)warp * ce_stage_warp(EPI);
        uint32_t use = 0;   // accumulators drained
        // (a warp gives up as a whole: its loads and stores are instructions of all lanes)
        // the common factor of the tokens' weights: left out of dz, put on its products
        float common = 1.f;
        if (EPI != kCeStats && a.weights != nullptr) common = ce_largest_weight(a, &s_weight);
        if ((EPI == kCeDz || EPI == kCeDz3) && a.rows_out != nullptr) ce_rows_of_h(a, warp, lane);
        if (GRADS && a.total != nullptr && a.total[1] > 0.f) common = 1.f / a.total[1];
        for (int k = 0; !__any_sync(0xffffffffu, *abort_flag) && ce_item(a, GRADS, pair, pairs, k, rank, it); ++k, ++use) {
            const CeSide& c0 = a.c[it.side];
            const uint32_t buf = use & 1u;
            // what a row needs besides its logits is fetched while the tile is computed
            float wgt = 0.f, lse2 = 0.f;
            long long tgt = -1;
            if (EPI == kCeDz || EPI == kCeDz3) {
                const int t = it.m0 + row;
                if (t < c0.M) {
                    const long long tg = a.target[t];
                    tgt = tg - c0.b_row - (long long)it.nt * kCeN;
                    // a row without a valid target adds nothing to the gradients
                    if (tg >= 0 && tg < a.V)
                        wgt = a.dloss != nullptr ? a.dloss[t] : a.weights != nullptr ? ce_ratio(a.weights[t], common) : 1.f;
                    lse2 = a.lse[t] * kLog2e;
                }
            }
            const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
            float sum[kCeN / 2];   // (CHAINS)
            if (CHAINS) {
                // each accumulator holds at most kChain stages; they add up in registers
#pragma unroll
                for (int j = 0; j < kCeN / 2; ++j) sum[j] = 0.f;
                bool lost = false;
                for (int k0 = it.k0; k0 < it.k1; k0 += kChain, ++use) {
                    const uint32_t b = use & 1u;
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_acc[b], (use >> 1) & 1u))) {
                        lost = true;
                        break;
                    }
                    tmem_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < kCeN / 2; c += 32) {
                        float v[2][16];
                        ce_columns(lanes + b * (uint32_t)kCeN + hf * (kCeN / 2) + (uint32_t)c, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c + j] += v[j / 16][j % 16];
                    }
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_map(&s_free[b], 0));
                }
                if (lost) {
                    if (lane == 0) fail();
                    break;
                }
                --use;   // the loop over the items counts the last one
            } else {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_acc[buf], (use >> 1) & 1u))) {
                    if (lane == 0) fail();
                    break;
                }
                tmem_fence_after_sync();
            }
            const uint32_t taddr = lanes + buf * (uint32_t)kCeN;   // (not CHAINS)
            if (EPI == kCeStats) {
                ce_epi_stats<CAP, CHAINS>(a, it, row, taddr, hf, sum);
            } else if (EPI == kCeGrads3) {
#pragma unroll
                for (int c = 0; c < kCeN / 2; c += 32)
                    ce_store_f32(tm.s[it.side], c0, it, &sum[c], common, stg, hf * (kCeN / 2) + c, q4, lane);
            } else if (GRADS && c0.part != nullptr) {
                for (int c = hf * (kCeN / 2); c < (hf + 1) * (kCeN / 2); c += 32) {
                    float v[2][16];
                    ce_columns(taddr + (uint32_t)c, v);
                    ce_store_f32(tm.s[it.side], c0, it, &v[0][0], common, stg, c, q4, lane);
                }
            } else {
                // BF16 results by TMA stores from swizzled staging, 32 columns at a time
                constexpr bool PARTS = EPI == kCeDz3;
                const int y = c0.s_row + it.m0 + 32 * q4;
                const bool store = it.m0 + 32 * q4 < c0.M;   // rows past the matrix are clipped by the TMA
                const int nv = c0.N - it.nt * kCeN;                 // columns of this tile inside the matrix
#pragma unroll 1
                for (int c = hf * (kCeN / 2); c < (hf + 1) * (kCeN / 2); c += 32) {
                    float v[2][16];
                    if (CHAINS)
                        ce_take(sum, v);
                    else
                        ce_columns(taddr + (uint32_t)c, v);
                    if (EPI == kCeDz || EPI == kCeDz3) {
                        if (CAP) ce_tanh(a, v);
                        const bool mine = tgt >= c && tgt < c + 32;   // a lane in many
                        float one = wgt;   // what the target's 1 becomes
                        if (CAP && mine) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (tgt == c + j) one = wgt * fmaf(-v[j / 16][j % 16], v[j / 16][j % 16], 1.f);
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float th = v[j / 16][j % 16];   // (the logit itself without a cap)
                            float e = ex2_approx(fmaf(th, CAP ? a.softcap * kLog2e : kLog2e, -lse2));
                            e *= wgt;
                            if (CAP) e *= fmaf(-th, th, 1.f);
                            v[j / 16][j % 16] = e;
                        }
                        if (mine) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (tgt == c + j) v[j / 16][j % 16] -= one;
                        }
                        if (c + 32 > nv) {   // past the vocabulary
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c + j >= nv) v[j / 16][j % 16] = 0.f;
                        }
                        // a row without a weight has exact zeros (its lse may be anything)
                        if (wgt == 0.f) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j / 16][j % 16] = 0.f;
                        }
                    }
                    if (GRADS) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j / 16][j % 16] *= common;
                    }
                    if (PARTS) {
                        // each part is what BF16 holds of what the ones before it left (24 bits in all)
                        const int x = it.nt * kCeN + c;
#pragma unroll
                        for (int p = 0; p < kCeParts; ++p) {
                            const int box = (p + (c / 32) * kCeParts) & 1;   // the two boxes in turns
                            if (lane == 0) bulk_wait_read<1>();              // the store before the last has read it
                            __syncwarp();
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int pu = u ^ ((lane >> 1) & 3);
                                float* e = v[u >> 1] + 8 * (u & 1);
                                const uint4 q = pack8(e);
                                *reinterpret_cast<uint4*>(stg + (size_t)box * kCeBox + (size_t)lane * 64 + 16 * pu) = q;
                                if (p + 1 < kCeParts) {
                                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float2 f = bf2_to_f2(w[k]);
                                        e[2 * k] -= f.x;
                                        e[2 * k + 1] -= f.y;
                                    }
                                }
                            }
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) {
                                if (store && x < c0.s_cols)
                                    tma_store_2d(p == 0 ? &tm.s[it.side] : &tm.more[p == 2], x, y,
                                                 stg + (size_t)box * kCeBox);
                                bulk_commit();   // (an empty group keeps the count)
                            }
                        }
                        continue;
                    }
                    const bool second = (c & 32) != 0;   // of a wide box
                    if (!second && lane == 0) bulk_wait_read<0>();   // the box is read out
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int pu = (u + (second ? 4 : 0)) ^ (lane & 7);
                        *reinterpret_cast<uint4*>(stg + (size_t)lane * 128 + 16 * pu) = pack8(v[u >> 1] + 8 * (u & 1));
                    }
                    if (!second) continue;
                    fence_proxy_async();
                    __syncwarp();
                    const int x = it.nt * kCeN + c - 32;
                    if (lane == 0 && store && x < c0.s_cols) {
                        tma_store_2d(&tm.s[it.side], x, y, stg);
                        bulk_commit();
                    }
                }
            }
            if (CHAINS) continue;   // the accumulators are free already
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_map(&s_free[buf], 0));
        }
        if (lane == 0) bulk_wait_all();   // every store has completed before the CTA may exit
    }
    __syncthreads();
    cluster_sync();   // neither CTA leaves, or gives its columns back, while the other may still use them
    if (warp == kCeIssuer) {
        tmem_fence_after_sync();
        tmem_dealloc2(tmem, kCeTmemCols);
    }
    cluster_sync();
}

// (m, s) of a row over two sets of columns.
__device__ __forceinline__ float2 ce_join(float2 p, float2 q) {
    const float m = fmaxf(p.x, q.x);
    const float ref = m == -INFINITY ? 0.f : m;
    return make_float2(m, p.y * ex2_approx((p.x - ref) * kLog2e) + q.y * ex2_approx((q.x - ref) * kLog2e));
}

// The statistics of a few tokens (T <= 4, RT = T rounded up to a power of two):
// every row of w is read once by one warp, so the kernel is bound by reading w,
// where the tensor-core tiles would spend the time of 256 rows on them and have
// too few tiles to share out (one token, 32768 x 1024: see launch_ce_few).
// A warp takes a run of rows, R at a time, a lane 8 channels of each (16
// bytes); the tokens' channels come from shared memory, once for the R rows.
// R T sums over the lanes end in one lane each by halving exchanges, and each
// lane keeps its own running (max, sum), joined over the CTA at the end.
template <int RT, int R>
__global__ void __launch_bounds__(256, kCeFewThreads / 256 / (RT == 1 ? 1 : 2)) ce_few_kernel(const uint4* __restrict__ h, const uint4* __restrict__ w, int T,
                                                     const CeGemmArgs a) {
    constexpr int NA = RT * R;
    static_assert(NA <= 32, "one lane a sum");
    extern __shared__ __align__(16) uint4 sh[];   // [T][D / 8]
    __shared__ float2 red[8][NA];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = a.c[0].K / 8, V = a.c[0].N;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.status[0] = a.status[1] = 0u;
    for (int i = threadIdx.x; i < T * nv; i += 256) sh[i] = __ldg(h + i);
    __syncthreads();
    const long long id = (long long)blockIdx.x * 8 + warp, n = (long long)gridDim.x * 8;
    const int v0 = (int)(V * id / n), v1 = (int)(V * (id + 1) / n);
    // this lane's sum is (row r, token t); the lanes past NA repeat others'
    const int t = lane % RT, r = (lane / RT) % R;
    const long long tgt = t < T ? a.target[t] : -1;
    float mx = -INFINITY, sum = 0.f;
    for (int v = v0; v < v1; v += R) {
        float acc[NA];
#pragma unroll
        for (int i = 0; i < NA; ++i) acc[i] = 0.f;
#pragma unroll 2
        for (int c = lane; c < nv; c += 32) {
            uint4 q[R];
#pragma unroll
            for (int i = 0; i < R; ++i)
                q[i] = v + i < v1 ? __ldcs(w + (size_t)(v + i) * nv + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const uint4 x = sh[(RT == 1 || j < T ? j : 0) * nv + c];
                const float2 x0 = bf2_to_f2(x.x), x1 = bf2_to_f2(x.y), x2 = bf2_to_f2(x.z), x3 = bf2_to_f2(x.w);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float2 y0 = bf2_to_f2(q[i].x), y1 = bf2_to_f2(q[i].y), y2 = bf2_to_f2(q[i].z),
                                 y3 = bf2_to_f2(q[i].w);
                    float s = acc[i * RT + j];
                    s = fmaf(x0.x, y0.x, s);
                    s = fmaf(x0.y, y0.y, s);
                    s = fmaf(x1.x, y1.x, s);
                    s = fmaf(x1.y, y1.y, s);
                    s = fmaf(x2.x, y2.x, s);
                    s = fmaf(x2.y, y2.y, s);
                    s = fmaf(x3.x, y3.x, s);
                    s = fmaf(x3.y, y3.y, s);
                    acc[i * RT + j] = s;
                }
            }
        }
        // halving exchanges: lane l ends with the sum of index l % NA over all lanes
#pragma unroll
        for (int k = NA / 2; k >= 1; k >>= 1) {
            const bool up = (lane & k) != 0;
#pragma unroll
            for (int i = 0; i < k; ++i) {
                const float give = up ? acc[i] : acc[i + k], keep = up ? acc[i + k] : acc[i];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, k);
            }
        }
        float z = acc[0];
#pragma unroll
        for (int k = NA; k < 32; k <<= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
        if (a.softcap > 0.f) z = ce_cap(a, z);
        if (t < T && v + r < v1) {
            if (tgt == v + r && lane < NA) a.zt[t] = z;
            const float m = fmaxf(mx, z), ref = m == -INFINITY ? 0.f : m;
            sum = fmaf(sum, ex2_approx((mx - ref) * kLog2e), ex2_approx((z - ref) * kLog2e));
            mx = m;
        }
    }
    if (lane < NA) red[warp][lane] = make_float2(mx, sum);
    __syncthreads();
    if (warp == 0 && lane < T) {
        float2 p = make_float2(-INFINITY, 0.f);
        for (int k = 0; k < 8; ++k)
            for (int i = 0; i < R; ++i) p = ce_join(p, red[k][i * RT + lane]);
        a.stats[(size_t)blockIdx.x * T + lane] = p;
    }
}

// The sum of the losses (in two floats) and the number of rows counted over a
// CTA of WARPS warps, in a fixed order; the result in thread 0.
template <int WARPS>
__device__ __forceinline__ void ce_cta_total(TwoSum& s, int& n, float2* red, int* red_n) {
    s = warp_sum(s);
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        red[threadIdx.x >> 5] = make_float2(s.hi, s.lo);
        red_n[threadIdx.x >> 5] = n;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    s = TwoSum();
    n = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        s.add(red[w].x, red[w].y);
        n += red_n[w];
    }
}

// Rows' statistics joined over their `parts` column blocks, in a fixed order:
// a CTA takes kCeRows consecutive rows, thread (row, group) the parts group,
// group + kCeGroups, ...; then lse, loss, and the CTA's (sum of losses, number
// of rows counted).  The last CTA to finish adds the CTAs' sums in order.
// A target outside [0, V) is not counted; one past V sets the status word.
template <int ROWS>
__global__ void __launch_bounds__(256) ce_rows_kernel(const float2* __restrict__ stats, const float* __restrict__ zt,
                                                      const int64_t* __restrict__ target, int parts, int T, int V,
                                                      float* __restrict__ loss, float* __restrict__ lse,
                                                      int4* __restrict__ sums, float* __restrict__ total,
                                                      uint32_t* ticket, uint32_t* status) {
    constexpr int GROUPS = 256 / ROWS;
    __shared__ float2 red[GROUPS][ROWS];
    __shared__ float2 tot[8];
    __shared__ int tot_n[8];
    __shared__ bool last;
    pdl_trigger();
    pdl_wait();
    const int r = threadIdx.x % ROWS, g = threadIdx.x / ROWS;
    const int t = blockIdx.x * ROWS + r;
    float2 p = make_float2(-INFINITY, 0.f);
    if (t < T) {
        // eight parts at a time: their loads together, one maximum, independent exponentials
        for (int i = g; i < parts; i += 8 * GROUPS) {
            float2 q[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                q[k] = i + k * GROUPS < parts ? __ldcg(stats + (size_t)(i + k * GROUPS) * T + t) : make_float2(-INFINITY, 0.f);
            float m = p.x;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, q[k].x);
            const float ref = m == -INFINITY ? 0.f : m;
            float s = p.y * ex2_approx((p.x - ref) * kLog2e);
#pragma unroll
            for (int k = 0; k < 8; ++k) s = fmaf(q[k].y, ex2_approx((q[k].x - ref) * kLog2e), s);
            p = make_float2(m, s);
        }
    }
    red[g][r] = p;
    __syncthreads();
    for (int k = GROUPS / 2; k >= 1; k >>= 1) {
        if (g < k) red[g][r] = ce_join(red[g][r], red[g + k][r]);
        __syncthreads();
    }
    TwoSum sum;
    int n = 0;
    if (g == 0 && t < T) {
        p = red[0][r];
        const float l = p.x + logf(p.y);
        const long long tg = target[t];
        const bool counted = tg >= 0 && tg < V;
        if (tg >= V) atomicOr(status, kStatusTarget);
        sum.hi = counted ? l - __ldcg(zt + t) : 0.f;
        n = counted ? 1 : 0;
        lse[t] = l;
        loss[t] = sum.hi;
    }
    ce_cta_total<8>(sum, n, tot, tot_n);
    if (threadIdx.x == 0) {
        sums[blockIdx.x] = make_int4(__float_as_int(sum.hi), __float_as_int(sum.lo), n, 0);
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = TwoSum();
    n = 0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 256) {
        const int4 q = __ldcg(sums + i);
        sum.add(__int_as_float(q.x), __int_as_float(q.y));
        n += q.z;
    }
    ce_cta_total<8>(sum, n, tot, tot_n);
    if (threadIdx.x == 0) {
        total[0] = sum.value();
        total[1] = (float)n;
        *ticket = 0u;
    }
}

// The same for few rows and parts (T <= 256, T parts <= kCeRowsSmall) in one
// CTA: no ticket, fence and second look at the sums (with the statistics, 20
// tokens x 500 entries at D 128 13.0 -> 10.5 us, 8.3 without FP64 in the sums;
// from about 8000 rows x parts on, more CTAs are faster).  Thread (row, group)
// as above, a power of two of rows.
constexpr int kCeRowsSmall = 4096;
__global__ void __launch_bounds__(1024) ce_rows_small_kernel(const float2* __restrict__ stats,
                                                             const float* __restrict__ zt,
                                                             const int64_t* __restrict__ target, int parts, int T,
                                                             int rows, int V, float* __restrict__ loss,
                                                             float* __restrict__ lse, float* __restrict__ total,
                                                             uint32_t* status) {
    __shared__ float2 red[1024];
    __shared__ float2 tot[8];
    __shared__ int tot_n[8];
    const int t = threadIdx.x & (rows - 1), g = threadIdx.x / rows, groups = 1024 / rows;
    pdl_trigger();
    pdl_wait();
    const long long tg = g == 0 && t < T ? target[t] : -1;
    const bool counted = tg >= 0 && tg < V;
    float2 p = make_float2(-INFINITY, 0.f);
    if (t < T)
        for (int i = g; i < parts; i += groups) p = ce_join(p, __ldcg(stats + (size_t)i * T + t));
    const float zt_t = counted ? __ldcg(zt + t) : 0.f;
    // the groups of a row inside a warp, then over the warps
    for (int o = rows; o < 32; o <<= 1) {
        const float2 q = make_float2(__shfl_xor_sync(0xffffffffu, p.x, o), __shfl_xor_sync(0xffffffffu, p.y, o));
        p = threadIdx.x & o ? ce_join(q, p) : ce_join(p, q);   // the same order in both lanes
    }
    red[threadIdx.x] = p;
    __syncthreads();
    TwoSum sum;
    int n = 0;
    if (g == 0 && t < T) {
        const int step = rows < 32 ? 32 : rows;
        for (int i = t + step; i < 1024; i += step) p = ce_join(p, red[i]);
        const float l = p.x + logf(p.y);
        if (tg >= V) atomicOr(status, kStatusTarget);
        sum.hi = counted ? l - zt_t : 0.f;
        n = counted ? 1 : 0;
        lse[t] = l;
        loss[t] = sum.hi;
    }
    // the rows are in the first eight warps
    if (threadIdx.x >= 256) {
        __syncthreads();
        __syncthreads();
        return;
    }
    ce_cta_total<8>(sum, n, tot, tot_n);
    if (threadIdx.x == 0) {
        total[0] = sum.value();
        total[1] = (float)n;
    }
}

// out[i] = sum of part[p][i] over p in order, as FP32 or BF16; n a multiple of 4.
template <bool F32>
__global__ void __launch_bounds__(256) ce_sum_kernel(const float4* __restrict__ part, long long stride4, int parts,
                                                     long long n4, void* __restrict__ out) {
    pdl_trigger();
    pdl_wait();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long long)gridDim.x * 256) {
        float4 s = __ldcg(part + i);
        for (int p = 1; p < parts; ++p) {
            const float4 v = __ldcg(part + (size_t)p * stride4 + i);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        if (F32)
            static_cast<float4*>(out)[i] = s;
        else
            static_cast<uint2*>(out)[i] = make_uint2(f2_to_bf2(s.x, s.y), f2_to_bf2(s.z, s.w));
    }
}

// 2-D map over a row-major BF16 matrix [rows][cols] with row stride ld.
bool ce_map(CUtensorMap* map, const void* ptr, long long cols, long long rows, long long ld, int box_cols,
            int box_rows, CUtensorMapSwizzle sw) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand's map: 128 rows of two 64-column chunks in one box (the columns
// seen as [cols / 64] chunks, `whole`), or of one chunk.
bool ce_operand(CUtensorMap* map, const void* ptr, long long cols, long long rows, long long ld, bool whole,
                int box_rows = 128) {
    if (!whole) return ce_map(map, ptr, cols, rows, ld, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
    cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 2};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An FP32 result's map: [splits][rows][cols] in boxes of 32 x 32.
bool ce_result_f32(CUtensorMap* map, const CeSide& c) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)c.N, (cuuint64_t)c.M, (cuuint64_t)c.splits};
    cuuint64_t strides[2] = {(cuuint64_t)c.N * 4, (cuuint64_t)c.M * (cuuint64_t)c.N * 4};
    cuuint32_t box[3] = {32, 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, c.part, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A BF16 result's map: the store boxes.
bool ce_result(CUtensorMap* map, const void* ptr, long long cols, long long rows, long long ld, bool wide) {
    return ce_map(map, ptr, cols, rows, ld, wide ? 64 : 32, 32, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Rows of a box of K-major A: with few tokens only as many as there are, in whole
// swizzle atoms (a box mostly outside the matrix takes as long to fill with
// zeros: 16 tokens x 32768 entries at D 1024, 26.6 -> 22.7 us).
int ce_a_rows(int M) { return std::min(128, (M + 7) / 8 * 8); }
// What an item of dh or dw costs, in K steps: its own, or its epilogue's if that is longer.
constexpr int kCeEpiSteps = 4;
int ce_item_steps(const CeSide& c) { return std::max(kCeEpiSteps, c.ksteps / c.splits); }
int ce_pairs() { return std::max(1, block_gemm_sms() / 2); }

template <int EPI, bool CAP, bool CHAINS>
cudaError_t ce_launch(const CeMaps& tm, CeGemmArgs& a, cudaStream_t s, bool pdl) {
    auto* fn = ce_gemm_kernel<EPI, CAP, CHAINS>;
    constexpr size_t smem = ce_smem(EPI);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kCeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // once per device: the shared memory, and as many pairs as fit at once (the
    // query is slow next to a launch)
    static std::atomic<int> cached[64];
    int dev = 0;
    const cudaError_t de = cudaGetDevice(&dev);
    if (de != cudaSuccess) return de;
    const bool keep = dev >= 0 && dev < 64;
    int pairs = keep ? cached[dev].load(std::memory_order_acquire) : 0;
    if (pairs < 1) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2);
        if (cudaOccupancyMaxActiveClusters(&pairs, fn, &cfg) != cudaSuccess || pairs < 1) pairs = ce_pairs();
        if (keep) cached[dev].store(pairs, std::memory_order_release);
    }
    pairs = std::min(pairs, a.c[0].n_items + a.c[1].n_items);
    cfg.gridDim = dim3(2u * (unsigned)pairs);
    // the pairs left with one dh item less make up for its K steps in dw items
    a.extra = 0;
    if ((EPI == kCeGrads || EPI == kCeGrads3) && a.c[0].n_items % pairs != 0)
        a.extra = (2 * ce_item_steps(a.c[0]) + ce_item_steps(a.c[1])) / (2 * ce_item_steps(a.c[1]));
    if (pdl) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, fn, tm, a);
}

}  // namespace

int ce_m_tiles(long long M) { return (int)((M + kCeM - 1) / kCeM); }
int ce_n_tiles(long long N) { return (int)((N + kCeN - 1) / kCeN); }

// Splits of the K axes of dh [T][D] (K = the piece of V) and dw [piece][D]
// (K = T), `parts` times as long: no item longer than a pair's
// share of all the steps (or 8 steps), so that a long axis with few tiles
// around it is spread over the pairs.
void ce_grad_splits(long long T, long long V, long long D, int parts, int sms, int* h_splits, int* w_splits) {
    const long long ch = parts * ((V + kCeK - 1) / kCeK), cw = parts * ((T + kCeK - 1) / kCeK);
    const long long e = kCeEpiSteps;
    const long long steps =
        ((long long)ce_m_tiles(T) * std::max(e, ch) + (long long)ce_m_tiles(V) * std::max(e, cw)) * ce_n_tiles(D);
    const long long most = std::max(8LL, steps / std::max(1, sms / 2));
    *h_splits = (int)std::min<long long>(kCeSplitsMax, (ch + most - 1) / most);
    *w_splits = (int)std::min<long long>(kCeSplitsMax, (cw + most - 1) / most);
}

namespace {

// Fills a contraction's tile counts.
void ce_side(CeSide& c, int parts) {
    c.m_tiles = ce_m_tiles(c.M);
    c.n_tiles = ce_n_tiles(c.N);
    c.part_steps = (c.K + kCeK - 1) / kCeK;
    c.ksteps = parts * c.part_steps;
    if (c.splits < 1) c.splits = 1;
    c.n_items = c.m_tiles * c.n_tiles * c.splits;
}

template <int EPI, bool CHAINS>
cudaError_t ce_logits_as(const CeMaps& tm, CeGemmArgs& a, cudaStream_t s, bool pdl) {
    return a.softcap > 0.f ? ce_launch<EPI, true, CHAINS>(tm, a, s, pdl) : ce_launch<EPI, false, CHAINS>(tm, a, s, pdl);
}

}  // namespace

// Logits of h [T][D] and rows a.c[0].b_row on of w [V][D]: their statistics,
// or dz [T][ldz] in `parts` parts (one, or kCeParts); ldz is a multiple of 64.
cudaError_t launch_ce_logits(const CeGemmArgs& in, const void* h, const void* w, int V, void* dz, int parts,
                             size_t part_bytes, long long ldz, cudaStream_t s, bool pdl) {
    CeGemmArgs a = in;
    CeSide& c = a.c[0];
    ce_side(c, 1);
    a.c[1].n_items = 0;
    CeMaps tm;
    a.whole = c.K % 64 == 0;
    const int rows = ce_a_rows(c.M);
    a.a_chunk = rows * 128;
    if (!ce_operand(&tm.a[0][0], h, c.K, c.M, c.K, a.whole, rows) || !ce_operand(&tm.b[0], w, c.K, V, c.K, a.whole))
        return cudaErrorInvalidValue;
    for (auto& row : tm.a) row[0] = row[1] = tm.a[0][0];
    tm.b[1] = tm.b[0];
    for (auto* m : {&tm.s[0], &tm.s[1], &tm.more[0], &tm.more[1]}) *m = tm.a[0][0];
    for (int p = 0; dz != nullptr && p < parts; ++p)
        if (!ce_result(p == 0 ? &tm.s[0] : &tm.more[p - 1], static_cast<char*>(dz) + p * part_bytes, c.s_cols, c.M, ldz,
                       parts == 1))
            return cudaErrorInvalidValue;
    // 32 MB of h per group of row tiles
    a.group = (int)std::max(1LL, std::min<long long>(c.m_tiles, (32LL << 20) / ((long long)c.K * 2 * kCeM)));
    // dz goes by the statistics' logits: their truncations meet in e^{z - lse} and mostly cancel
    bool chains = c.ksteps > ce_chain(kCeStats);
    if (dz != nullptr && parts > 1) {
        // (few tokens' statistics have none to cancel)
        chains = chains || (ce_is_few(c.M, c.K) && c.ksteps > ce_chain(kCeDz3));
        return chains ? ce_logits_as<kCeDz3, true>(tm, a, s, pdl) : ce_logits_as<kCeDz3, false>(tm, a, s, pdl);
    }
    if (dz != nullptr)
        return chains ? ce_logits_as<kCeDz, true>(tm, a, s, pdl) : ce_logits_as<kCeDz, false>(tm, a, s, pdl);
    return chains ? ce_logits_as<kCeStats, true>(tm, a, s, pdl) : ce_logits_as<kCeStats, false>(tm, a, s, pdl);
}

// The statistics of T <= 4 tokens, one part a CTA, as long as their rows fit.
// Events around the launch, w not in the L2, for 1, 2, 3 and 4 tokens (the
// tensor-core tiles, which take 5 and more: the last figure): 32768 x 1024 21, 21,
// 23, 23 (27) us; 32768 x 4096 56, 52, 62, 62 (70); 32768 x 8192 101, 93, 112, - (119);
// 5000 x 2048 21, 16, 15, 15 (23).
bool ce_is_few(int T, int D) { return T <= 4 && (size_t)T * D * 2 <= kCeFewSmem; }
int ce_few_parts(int T, int sms) { return kCeFewThreads / 256 / (T == 1 ? 1 : 2) * sms; }
cudaError_t launch_ce_few(const CeGemmArgs& a, const void* h, const void* w, cudaStream_t s, bool pdl) {
    const int T = a.c[0].M, D = a.c[0].K;
    const int kind = T == 1 ? 0 : T == 2 ? 1 : 2;
    auto* fn = kind == 0 ? ce_few_kernel<1, 8> : kind == 1 ? ce_few_kernel<2, 8> : ce_few_kernel<4, 4>;
    // with the kernel's own arrays this may pass the 48 KB that need no leave; asked for once per device
    static std::atomic<bool> allowed[3][64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < 64;
    if (!keep || !allowed[kind][dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kCeFewSmem);
        if (e != cudaSuccess) return e;
        if (keep) allowed[kind][dev].store(true, std::memory_order_release);
    }
    const size_t smem = (size_t)T * D * 2;
    return launch_ex(fn, dim3((unsigned)ce_few_parts(T, block_gemm_sms())), dim3(256), smem, s, pdl,
                     static_cast<const uint4*>(h), static_cast<const uint4*>(w), T, a);
}

// a.c[0]: dh [T][D] (+)= dz w's rows b_row on; a.c[1]: dw = dz^T h, rows s_row
// on of a matrix [V][D].  Each as FP32 into its `part`, or as BF16 into S.
cudaError_t launch_ce_grads(const CeGemmArgs& in, const void* dz, int parts, size_t part_bytes, long long ldz,
                            const void* h, const void* w, int V, void* dh, void* dw, cudaStream_t s, bool pdl) {
    CeGemmArgs a = in;
    ce_side(a.c[0], parts);
    ce_side(a.c[1], parts);
    const long long T = a.c[0].M, D = a.c[0].N;
    CeMaps tm;
    a.whole = D % 64 == 0;   // dz's own rows always are
    const int rows = ce_a_rows((int)T);
    a.a_chunk = rows * 128;
    for (int p = 0; p < kCeParts; ++p) {
        const void* part = static_cast<const char*>(dz) + (p < parts ? p : 0) * part_bytes;
        if (!ce_operand(&tm.a[p][0], part, ldz, T, ldz, true, rows) || !ce_operand(&tm.a[p][1], part, ldz, T, ldz, true))
            return cudaErrorInvalidValue;
    }
    if (!ce_operand(&tm.b[0], w, D, V, D, a.whole) || !ce_operand(&tm.b[1], h, D, T, D, a.whole))
        return cudaErrorInvalidValue;
    tm.more[0] = tm.more[1] = tm.a[0][0];
    if (!(a.c[0].part != nullptr ? ce_result_f32(&tm.s[0], a.c[0]) : ce_result(&tm.s[0], dh, D, T, D, true)) ||
        !(a.c[1].part != nullptr ? ce_result_f32(&tm.s[1], a.c[1]) : ce_result(&tm.s[1], dw, D, V, D, true)))
        return cudaErrorInvalidValue;
    if (parts > 1) return ce_launch<kCeGrads3, false, true>(tm, a, s, pdl);
    return ce_launch<kCeGrads, false, false>(tm, a, s, pdl);
}

// Rows per CTA of the statistics kernel: 32 (a warp reads 32 rows of one part),
// 8 or one where there are fewer rows and the parts are what there is to share
// out.
int ce_rows_per_cta(int T) { return T <= 256 ? 1 : T <= 8192 ? 8 : 32; }
int ce_row_ctas(int T) { return (T + ce_rows_per_cta(T) - 1) / ce_rows_per_cta(T); }

cudaError_t launch_ce_rows(const float2* stats, const float* zt, const int64_t* target, int parts, int T, int V,
                           float* loss, float* lse, int4* sums, float* total, uint32_t* ticket, uint32_t* status,
                           cudaStream_t s, bool pdl) {
    if (T <= 256 && (long long)T * parts <= kCeRowsSmall) {
        int pow2 = 1;
        while (pow2 < T) pow2 <<= 1;
        return launch_ex(ce_rows_small_kernel, dim3(1), dim3(1024), 0, s, pdl, stats, zt, target, parts, T, pow2, V, loss,
                         lse, total, status);
    }
    const int rows = ce_rows_per_cta(T);
    auto* fn = rows == 1 ? ce_rows_kernel<1> : rows == 8 ? ce_rows_kernel<8> : ce_rows_kernel<32>;
    return launch_ex(fn, dim3((unsigned)ce_row_ctas(T)), dim3(256), 0, s, pdl, stats, zt, target, parts, T, V, loss, lse,
                     sums, total, ticket, status);
}

cudaError_t launch_ce_sum(const float* part, long long stride, int parts, long long n, void* out, bool f32,
                          cudaStream_t s, bool pdl) {
    const long long blocks = std::max(1LL, std::min(8192LL, (n / 4 + 255) / 256));
    const float4* p = reinterpret_cast<const float4*>(part);
    if (f32)
        return launch_ex(ce_sum_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, pdl, p, stride / 4, parts, n / 4,
                         out);
    return launch_ex(ce_sum_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, pdl, p, stride / 4, parts, n / 4,
                     out);
}

}  // namespace lrs

// Embedding lookup with a scale, and its gradient by sorted tokens.
//
//   y_t = scale w[token_t]               (zeros for a negative token)
//   dw[v] = scale sum of dy_t over the tokens t with token_t = v, added in the tokens' order
//
// Bound by bandwidth.  The gradient has no atomic additions: the tokens are
// sorted (stably), the sorted list is cut into chunks of the same length, so
// that a frequent token costs as much per occurrence as a rare one, and the rows
// that reach over chunks are joined from partial sums in their order.
//   sort   `owners` CTAs, each with the vocabulary rows v = owner (mod owners):
//          frequent tokens, which lie side by side in most vocabularies, go to
//          different CTAs.  Each CTA looks through all the tokens (8 T bytes from
//          L2: no histogram or prefix crosses CTAs, one launch), counts its rows'
//          and all lower owners' tokens, and places its own in order.
//   sum    a CTA a chunk of sorted places, threads across the row; other CTAs zero
//          the rows without a token.
//   join   rows that reach over a chunk's end.
#include <algorithm>

#include "ssm.cuh"

namespace lrs {

namespace {

template <bool F32, int R>
__global__ void __launch_bounds__(256) embedding_fwd_kernel(const EmbedArgs a) {
    pdl_trigger();
    pdl_wait();
    const int nv = a.D / 8;
    const long long t0 = ((long long)blockIdx.x * blockDim.y + threadIdx.y) * R;
    long long tok[R];
#pragma unroll
    for (int r = 0; r < R; ++r) tok[r] = t0 + r < a.T ? __ldg(a.tokens + t0 + r) : -1;
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        uint4 q[R], q2[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            q[r] = q2[r] = make_uint4(0u, 0u, 0u, 0u);
            if (tok[r] < 0 || tok[r] >= a.V) continue;
            const uint4* p = static_cast<const uint4*>(a.w) + (tok[r] * nv + v) * (F32 ? 2 : 1);
            q[r] = __ldg(p);
            if (F32) q2[r] = __ldg(p + 1);
        }
        const f2x s = dup2(a.scale);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (t0 + r >= a.T) break;
            f2x o[4];
            if (F32) {
                o[0] = pk2(__uint_as_float(q[r].x), __uint_as_float(q[r].y));
                o[1] = pk2(__uint_as_float(q[r].z), __uint_as_float(q[r].w));
                o[2] = pk2(__uint_as_float(q2[r].x), __uint_as_float(q2[r].y));
                o[3] = pk2(__uint_as_float(q2[r].z), __uint_as_float(q2[r].w));
            } else {
                unpack_pairs(q[r], o);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = tok[r] < a.V ? mul2(o[e], s) : dup2(NAN);   // no such row
            reinterpret_cast<uint4*>(a.y)[(t0 + r) * nv + v] = make_uint4(x2bf(o[0]), x2bf(o[1]), x2bf(o[2]), x2bf(o[3]));
        }
    }
}

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRows = 4096;     // vocabulary rows of an owner, at most
constexpr int kSortList = 8192;     // tokens of an owner that it places from shared memory
constexpr int kOwners = 128;        // a power of two, as are the owners of larger vocabularies
constexpr int kEmbedChunk = 32;     // sorted places of a CTA of the sum

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const EmbedBwdArgs a, int rows) {
    extern __shared__ __align__(16) uint8_t buf[];
    int2* held = reinterpret_cast<int2*>(buf);              // [kSortList]
    int* hist = reinterpret_cast<int*>(held + kSortList);   // [rows]: counts, then the next free place of each row
    __shared__ int mine[kSortWarps], lower[kSortWarps], bad;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, own = blockIdx.x, owners = a.owners, shift = 31 - __clz(owners);
    for (int i = tid; i < rows; i += kSortThreads) hist[i] = 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    // a warp's tokens are consecutive
    const int per = ((a.T + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const long long begin = (long long)warp * per, end = min((long long)a.T, begin + per);
    int n = 0, less = 0;
#pragma unroll 4
    for (long long t = begin + lane; t < end; t += 32) {
        const long long v = __ldg(a.tokens + t);
        if (v < 0) continue;
        if (v >= a.V) {
            bad = 1;
            continue;
        }
        const int o = (int)v & (owners - 1);
        less += o < own;
        if (o == own) {
            ++n;
            atomicAdd(&hist[(int)v >> shift], 1);
        }
    }
    n = __reduce_add_sync(0xffffffffu, n);
    less = __reduce_add_sync(0xffffffffu, less);
    if (lane == 0) {
        mine[warp] = n;
        lower[warp] = less;
    }
    __syncthreads();
    int base = 0, before = 0, total = 0;   // places of lower owners, of this owner's earlier warps, of all its warps
    for (int w = 0; w < kSortWarps; ++w) {
        base += lower[w];
        if (w < warp) before += mine[w];
        total += mine[w];
    }
    // counts to first places, a run of rows a thread
    {
        __shared__ int sums[kSortWarps];
        const int run = (rows + kSortThreads - 1) / kSortThreads, r0 = tid * run;
        int s = 0;
        for (int i = r0; i < min(rows, r0 + run); ++i) s += hist[i];
        int inc = s;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, m);
            if (lane >= m) inc += o;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int at = base + inc - s;
        for (int w = 0; w < warp; ++w) at += sums[w];
        for (int i = r0; i < min(rows, r0 + run); ++i) {
            const int c = hist[i];
            hist[i] = at;
            a.first[(long long)own * rows + i] = at;
            at += c;
        }
    }
    if (tid == 0 && own == owners - 1) {
        a.first[(long long)owners * rows] = base + total;
        *a.count = base + total;
    }
    if (tid == 0 && own == 0) *a.status = bad ? kStatusTarget : 0u;
    // this owner's tokens in order, in the places that they will take
    int2* list = total <= kSortList ? held : a.list + base;
    int at = before;
#pragma unroll 4
    for (long long t = begin; t < end; t += 32) {
        const long long v = t + lane < end ? __ldg(a.tokens + t + lane) : -1;
        const bool hit = v >= 0 && v < a.V && ((int)v & (owners - 1)) == own;
        const uint32_t m = __ballot_sync(0xffffffffu, hit);
        if (hit) list[at + __popc(m & ((1u << lane) - 1u))] = make_int2((int)(t + lane), (int)v >> shift);
        at += __popc(m);
    }
    __syncthreads();
    if (warp != 0) return;
    // each to its row's next place: 32 at a time, equal rows in the order of their lanes
    int2 next = lane < total ? list[lane] : make_int2(0, 0);
    for (int i = 0; i < total; i += 32) {
        const bool on = i + lane < total;
        const int2 e = on ? next : make_int2(0, -1 - lane);
        if (i + 32 + lane < total) next = list[i + 32 + lane];
        const uint32_t same = __match_any_sync(0xffffffffu, e.y);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (on) {
            const int place = hist[e.y] + rank;
            a.place[place] = make_int2(e.x, own * rows + e.y);
        }
        __syncwarp();
        if (on && rank == 0) hist[e.y] += __popc(same);
        __syncwarp();
    }
}

// 8 columns of a row of dw: scale v, onto what is there (accumulate).
__device__ __forceinline__ void put_row(const EmbedBwdArgs& a, long long row, int v8, const f2x (&v)[4]) {
    const long long at = row * a.D + 8LL * v8;
    const f2x s = dup2(a.scale);
    f2x o[4] = {0ull, 0ull, 0ull, 0ull};
    if (a.f32) {
        float* p = static_cast<float*>(a.dw) + at;
        if (a.accumulate) read_pairs(p, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fma2(s, v[e], o[e]);
        store_pairs(p, o);
    } else {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dw) + at);
        if (a.accumulate) unpack_pairs(*p, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fma2(s, v[e], o[e]);
        *p = make_uint4(x2bf(o[0]), x2bf(o[1]), x2bf(o[2]), x2bf(o[3]));
    }
}
// Vocabulary row of a row in sorted order.
__device__ __forceinline__ long long vocabulary_row(const EmbedBwdArgs& a, int rows, int s) {
    return (long long)(s % rows) * a.owners + s / rows;
}

__global__ void __launch_bounds__(256) embedding_sum_kernel(const EmbedBwdArgs a, int rows, int chunks) {
    __shared__ int2 place[kEmbedChunk];
    pdl_trigger();
    pdl_wait();
    const int nv = a.D / 8;
    if ((int)blockIdx.x >= chunks) {
        // rows without a token: 32 looked up at a time, then written
        __shared__ uint32_t empty;
        const int all = a.owners * rows, step = (gridDim.x - chunks) * 32, words = nv * (a.f32 ? 2 : 1);
        for (int s0 = (blockIdx.x - chunks) * 32; s0 < all; s0 += step) {
            if (threadIdx.x < 32) {
                const int s = s0 + threadIdx.x;
                const uint32_t m = __ballot_sync(0xffffffffu, s < all && __ldcg(a.first + min(s, all)) == __ldcg(a.first + min(s + 1, all)) &&
                                                                  vocabulary_row(a, rows, s) < a.V);
                if (threadIdx.x == 0) empty = m;
            }
            __syncthreads();
            for (uint32_t m = empty; m != 0u; m &= m - 1u) {
                const long long row = vocabulary_row(a, rows, s0 + __ffs(m) - 1);
                uint4* p = reinterpret_cast<uint4*>(a.dw) + row * words;
                for (int v = threadIdx.x; v < words; v += blockDim.x) p[v] = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncthreads();
        }
        return;
    }
    const int i0 = blockIdx.x * kEmbedChunk, n = min(kEmbedChunk, __ldcg(a.count) - i0);
    if (n <= 0) return;
    if ((int)threadIdx.x < n) place[threadIdx.x] = __ldcg(a.place + i0 + threadIdx.x);
    __syncthreads();
    // what of the chunk's first and last row lies in other chunks
    const bool from = __ldcg(a.first + place[0].y) < i0, to = __ldcg(a.first + place[n - 1].y + 1) > i0 + n;
    const int head = place[0].y, tail = place[n - 1].y;
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        f2x s[4] = {0ull, 0ull, 0ull, 0ull};
        constexpr int AHEAD = 8;
        for (int i = 0; i < n; i += AHEAD) {
            uint4 q[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i + k < n) q[k] = __ldg(reinterpret_cast<const uint4*>(a.dy) + (long long)place[i + k].x * nv + v);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (i + k >= n) break;
                const int row = place[i + k].y;
                f2x d[4];
                unpack_pairs(q[k], d);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = add2(s[e], d[e]);
                if (i + k + 1 < n && place[i + k + 1].y == row) continue;
                // the row ends here, or the chunk does: slot 0 for a row from an earlier chunk, 1 for one that goes on
                if (row == head && from)
                    store_pairs(a.part + (2LL * blockIdx.x) * a.D + 8 * v, s);
                else if (row == tail && to)
                    store_pairs(a.part + (2LL * blockIdx.x + 1) * a.D + 8 * v, s);
                else
                    put_row(a, vocabulary_row(a, rows, row), v, s);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] = 0ull;
            }
        }
    }
}

// The row that begins in chunk blockIdx.x and goes on past it.
__global__ void __launch_bounds__(256) embedding_join_kernel(const EmbedBwdArgs a, int rows) {
    pdl_trigger();
    pdl_wait();
    const int nv = a.D / 8, count = __ldcg(a.count);
    const int end = (blockIdx.x + 1) * kEmbedChunk;
    if (end >= count) return;
    const int row = __ldcg(a.place + end - 1).y;
    const int begin = __ldcg(a.first + row), last = __ldcg(a.first + row + 1);
    if (last <= end || begin < end - kEmbedChunk) return;
    const int more = (last - 1) / kEmbedChunk;   // its last chunk
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        f2x s[4];
        read_pairs(a.part + (2LL * blockIdx.x + 1) * a.D + 8 * v, s);
#pragma unroll 4
        for (int c = blockIdx.x + 1; c <= more; ++c) {
            f2x d[4];
            read_pairs(a.part + 2LL * c * a.D + 8 * v, d);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = add2(s[e], d[e]);
        }
        put_row(a, vocabulary_row(a, rows, row), v, s);
    }
}

int lanes_of(int D) { return std::min(256, (D / 8 + 31) / 32 * 32); }

template <bool F32>
cudaError_t fwd_as(const EmbedArgs& a, cudaStream_t s, bool pdl) {
    const int x = lanes_of(a.D), y = 256 / x;
    const dim3 block((unsigned)x, (unsigned)y);
    // four rows a thread in flight, one where there are few
    if ((long long)a.T <= 4LL * 152 * y)
        return launch_ex(embedding_fwd_kernel<F32, 1>, dim3((unsigned)((a.T + y - 1) / y)), block, 0, s, pdl, a);
    return launch_ex(embedding_fwd_kernel<F32, 4>, dim3((unsigned)(((long long)a.T + 4 * y - 1) / (4 * y))), block, 0, s, pdl, a);
}

int owner_rows(const EmbedBwdArgs& a) { return (a.V + a.owners - 1) / a.owners; }

}  // namespace

int embed_owners(int V) {
    int n = kOwners;
    while ((long long)n * kSortRows < V) n *= 2;
    return n;
}
long long embed_chunks(long long T) { return (T + kEmbedChunk - 1) / kEmbedChunk; }

cudaError_t launch_embedding(const EmbedArgs& a, cudaStream_t s, bool pdl) {
    return a.w32 ? fwd_as<true>(a, s, pdl) : fwd_as<false>(a, s, pdl);
}
cudaError_t launch_embedding_sort(const EmbedBwdArgs& a, cudaStream_t s, bool pdl) {
    const int rows = owner_rows(a);
    constexpr size_t held = kSortList * sizeof(int2);
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(embedding_sort_kernel), held + kSortRows * sizeof(int), allowed);
    if (e != cudaSuccess) return e;
    return launch_ex(embedding_sort_kernel, dim3((unsigned)a.owners), dim3(kSortThreads), held + rows * sizeof(int), s, pdl, a, rows);
}
cudaError_t launch_embedding_sum(const EmbedBwdArgs& a, cudaStream_t s, bool pdl) {
    const int rows = owner_rows(a), chunks = (int)embed_chunks(a.T);
    const int zero = a.accumulate ? 0 : std::min((a.owners * rows + 31) / 32, 152 * 8);
    return launch_ex(embedding_sum_kernel, dim3((unsigned)(chunks + zero)), dim3((unsigned)lanes_of(a.D)), 0, s, pdl, a, rows, chunks);
}
cudaError_t launch_embedding_join(const EmbedBwdArgs& a, cudaStream_t s, bool pdl) {
    return launch_ex(embedding_join_kernel, dim3((unsigned)embed_chunks(a.T)), dim3((unsigned)lanes_of(a.D)), 0, s, pdl, a,
                     owner_rows(a));
}

}  // namespace lrs

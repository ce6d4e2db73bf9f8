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
//   sum    a CTA a chunk of 16 sorted places and 1024 columns; the parts of a row
//          that reaches over chunks are joined, in their order and 32 at a time, by
//          whichever of their CTAs is done last, and those sums by whichever group is
//          (one CTA for all parts: 65536 tokens of two rows 303 us, so 56); other CTAs
//          zero the rows without a token.
// 16384 tokens, 32768 x 1024: lookup 14 us (67 MB, 4.7 TB/s), with FP32 gradients sort 10,
// sum 37 (168 MB, 4.5 TB/s; 6 CTAs an SM, 5 with the registers that it would take: 65536
// tokens 65 us, so 62).  The sort is bound by its pass over the tokens and by what its
// busiest CTA finds (65536 tokens 29 us, none frequent 15; with a lane after the other in
// place of whole warps where a token is frequent 47).
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

constexpr int kSortWarps = 32;
constexpr int kSortRows = 1024;     // vocabulary rows of an owner, at most
constexpr int kSortNotes = 96;      // tokens that a warp notes, 31 + 64 at least
constexpr int kSortAhead = 4;       // times 64 tokens that it asks for at once
constexpr int kOwners = 128;        // a power of two, as are the owners of larger vocabularies
constexpr int kEmbedChunk = 16;     // sorted places of a CTA of the sum
constexpr int kJoin = 32;           // parts of a row that one CTA joins
constexpr int kSumThreads = 128;    // of it, 8 columns each

// N times 64 tokens from t on (counted from a 16-byte boundary, `odd` before the array), two a lane and step, as {low, high}
// words; -1 from `end` on and outside the array.  All are asked for before one is used.
template <int N>
__device__ __forceinline__ void load_tokens(const EmbedBwdArgs& a, long long t, long long end, int odd, int lane, int4 (&q)[N]) {
    const int2* p = reinterpret_cast<const int2*>(a.tokens) - odd;
    bool cut = false;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const long long i = t + 64 * u + 2 * lane;
        const bool whole = i >= odd && i + 1 < end;
        cut |= !whole;
        q[u] = make_int4(-1, -1, -1, -1);
        if (whole) q[u] = __ldg(reinterpret_cast<const int4*>(p + i));
    }
    if (!cut) return;
#pragma unroll
    for (int u = 0; u < N; ++u) {   // the array's first and last token may lie alone in their pair
        const long long i = t + 64 * u + 2 * lane;
        if (i < odd && i + 1 < end) {
            const int2 v = __ldg(p + i + 1);
            q[u].z = v.x;
            q[u].w = v.y;
        } else if (i >= odd && i + 1 == end) {
            const int2 v = __ldg(p + i);
            q[u].x = v.x;
            q[u].y = v.y;
        }
    }
}

// Which of two tokens are this owner's; how many a lower owner's; whether one has no row.
struct Hits {
    bool h0, h1, past;
    int less;
};
__device__ __forceinline__ Hits hits_of(int4 q, uint32_t V, int own, int owners) {
    const bool in0 = q.y == 0 && (uint32_t)q.x < V, in1 = q.w == 0 && (uint32_t)q.z < V;
    const int o0 = q.x & (owners - 1), o1 = q.z & (owners - 1);
    return {in0 && o0 == own, in1 && o1 == own, (q.y >= 0 && !in0) || (q.w >= 0 && !in1), (in0 && o0 < own) + (in1 && o1 < own)};
}
// A warp takes consecutive tokens, so that a stable sort needs no order between
// threads: it counts its tokens of each row, a row's counts are added up over the
// warps, and the warp places its tokens from there on.  What it finds (one token of
// 128 is this owner's) it notes, to go through the tokens once; where that is more
// than it has room for (a frequent token's), it looks for them again.
__global__ void __launch_bounds__(kSortWarps * 32) embedding_sort_kernel(const EmbedBwdArgs a, int rows, int dones) {
    extern __shared__ __align__(16) int count[];   // [kSortWarps][rows], then each warp's next place in a row
    __shared__ int2 noted[kSortWarps][kSortNotes];
    __shared__ int lower[kSortWarps], sums[kSortWarps], bad;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, own = blockIdx.x, owners = a.owners, shift = 31 - __clz(owners);
    for (int i = tid; i < kSortWarps * rows; i += kSortWarps * 32) count[i] = 0;
    if (tid == 0) bad = 0;
    for (int i = own * kSortWarps * 32 + tid; i < dones; i += owners * kSortWarps * 32) a.done[i] = 0;
    __syncthreads();
    int* mine = count + warp * rows;
    // tokens are read in pairs on 16-byte boundaries; `odd`: the first pair begins one before the array
    const int odd = (int)(reinterpret_cast<uintptr_t>(a.tokens) >> 3 & 1u);
    const long long all = (long long)a.T + odd, per = (all + kSortWarps * 64 - 1) / (kSortWarps * 64) * 64;
    const long long begin = warp * per, end = min(all, begin + per);
    const uint32_t V = (uint32_t)a.V, before_me = (1u << lane) - 1u;
    int less = 0, found = 0;
    bool past = false;
    for (long long t = begin; t < end; t += 64 * kSortAhead) {
        int4 qs[kSortAhead];
        load_tokens(a, t, end, odd, lane, qs);
#pragma unroll
        for (int u = 0; u < kSortAhead; ++u) {
            const int4 q = qs[u];
            const Hits h = hits_of(q, V, own, owners);
            past |= h.past;
            less += h.less;
            const bool hit0 = h.h0, hit1 = h.h1;
            const uint32_t m0 = __ballot_sync(0xffffffffu, hit0), m1 = __ballot_sync(0xffffffffu, hit1);
            if ((m0 | m1) == 0u) continue;
            const int at = found + __popc(m0 & before_me) + __popc(m1 & before_me);
            const int pos = (int)(t - odd) + 64 * u + 2 * lane;
            if (hit0) {
                atomicAdd(&mine[q.x >> shift], 1);
                if (at < kSortNotes) noted[warp][at] = make_int2(pos, q.x >> shift);
            }
            if (hit1) {
                atomicAdd(&mine[q.z >> shift], 1);
                if (at + hit0 < kSortNotes) noted[warp][at + hit0] = make_int2(pos + 1, q.z >> shift);
            }
            found += __popc(m0) + __popc(m1);
        }
    }
    if (past) bad = 1;
    less = __reduce_add_sync(0xffffffffu, less);
    if (lane == 0) lower[warp] = less;
    __syncthreads();
    // a thread a row: the row's tokens, and where its first one goes
    int n = 0;
    if (tid < rows)
        for (int w = 0; w < kSortWarps; ++w) n += count[w * rows + tid];
    int inc = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    // places before: the lower owners', and the warps' before
    const int before = __reduce_add_sync(0xffffffffu, lower[lane] + (lane < warp ? sums[lane] : 0));
    int at = before + inc - n;
    if (tid < rows) {
        a.first[(long long)own * rows + tid] = at;
        if (own == owners - 1 && tid == rows - 1) {
            a.first[(long long)owners * rows] = at + n;
            *a.count = at + n;
        }
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = count[w * rows + tid];
            count[w * rows + tid] = at;
            at += c;
        }
    }
    if (tid == 0 && own == 0) *a.status = bad ? kStatusTarget : 0u;
    __syncthreads();
    // equal rows in the order of their lanes
    const auto put = [&](bool on, int2 e) {
        if (!on) e.y = -1 - lane;
        const uint32_t same = __match_any_sync(0xffffffffu, e.y);
        if (on) a.place[mine[e.y] + __popc(same & before_me)] = make_int2(e.x, own * rows + e.y);
        __syncwarp();
        if (on && (same & before_me) == 0u) mine[e.y] += __popc(same);
        __syncwarp();
    };
    int2* note = noted[warp];
    if (found <= kSortNotes) {
        for (int i = 0; i < found; i += 32) put(i + lane < found, note[min(i + lane, kSortNotes - 1)]);
        return;
    }
    int kept = 0;
    for (long long t = begin; t < end; t += 64 * kSortAhead) {
        int4 qs[kSortAhead];
        load_tokens(a, t, end, odd, lane, qs);
#pragma unroll 1
        for (int u = 0; u < kSortAhead; ++u) {
            const int4 q = qs[0];
#pragma unroll
            for (int k = 0; k + 1 < kSortAhead; ++k) qs[k] = qs[k + 1];
            const Hits h = hits_of(q, V, own, owners);
            const uint32_t m0 = __ballot_sync(0xffffffffu, h.h0), m1 = __ballot_sync(0xffffffffu, h.h1);
            const int at = kept + __popc(m0 & before_me) + __popc(m1 & before_me), pos = (int)(t - odd) + 64 * u + 2 * lane;
            if (h.h0) note[at] = make_int2(pos, q.x >> shift);
            if (h.h1) note[at + h.h0] = make_int2(pos + 1, q.z >> shift);
            kept += __popc(m0) + __popc(m1);
            if (kept < 32) continue;
            // whole warps of notes go to their places, the rest (31 at most, and 64 come with the next tokens) to the front
            __syncwarp();
            int i = 0;
            for (; i + 32 <= kept; i += 32) put(true, note[i + lane]);
            kept -= i;
            const int2 e = note[i + min(lane, kSortNotes - 1 - i)];
            __syncwarp();
            if (lane < kept) note[lane] = e;
            __syncwarp();
        }
    }
    __syncwarp();
    put(lane < kept, note[lane]);
}

// 8 columns of a row of dw (`old`: what they hold where the gradient is added to it).
struct Old {
    uint4 q[2];
};
__device__ __forceinline__ Old old_row(const EmbedBwdArgs& a, long long row, int v8) {
    Old o;
    o.q[0] = o.q[1] = make_uint4(0u, 0u, 0u, 0u);
    if (!a.accumulate) return o;
    const uint4* p = static_cast<const uint4*>(a.dw) + (row * (a.D / 8) + v8) * (a.f32 ? 2 : 1);
    o.q[0] = p[0];
    if (a.f32) o.q[1] = p[1];
    return o;
}
__device__ __forceinline__ f2x word_pair(uint32_t lo, uint32_t hi) { return pk2(__uint_as_float(lo), __uint_as_float(hi)); }
__device__ __forceinline__ void put_row(const EmbedBwdArgs& a, long long row, int v8, const f2x (&v)[4], const Old& old) {
    const f2x s = dup2(a.scale);
    uint4* p = static_cast<uint4*>(a.dw) + (row * (a.D / 8) + v8) * (a.f32 ? 2 : 1);
    f2x o[4];
    if (a.f32) {
        o[0] = word_pair(old.q[0].x, old.q[0].y);
        o[1] = word_pair(old.q[0].z, old.q[0].w);
        o[2] = word_pair(old.q[1].x, old.q[1].y);
        o[3] = word_pair(old.q[1].z, old.q[1].w);
    } else {
        unpack_pairs(old.q[0], o);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fma2(s, v[e], o[e]);
    if (a.f32)
        put_pairs(reinterpret_cast<float*>(p), o);
    else
        *p = make_uint4(x2bf(o[0]), x2bf(o[1]), x2bf(o[2]), x2bf(o[3]));
}
// Vocabulary row of a row in sorted order.
__device__ __forceinline__ long long vocabulary_row(const EmbedBwdArgs& a, int rows, int s) {
    return (long long)(s % rows) * a.owners + s / rows;
}

// A row's parts: slot 1 of the chunk where it begins, slot 0 of those after it.
struct RowParts {
    int first, count;   // chunks
};
__device__ __forceinline__ RowParts parts_of(const EmbedBwdArgs& a, int row) {
    const int begin = __ldcg(a.first + row), last = __ldcg(a.first + row + 1);
    return {begin / kEmbedChunk, (last - 1) / kEmbedChunk - begin / kEmbedChunk + 1};
}

__device__ __forceinline__ float* part_at(const EmbedBwdArgs& a, const RowParts& r, int i, int v) {
    return a.part + (2LL * (r.first + i) + (i == 0 ? 1 : 0)) * a.D + 8 * v;
}
// s: the sum of the parts from, from + step, .. before to, in that order
__device__ __forceinline__ void add_parts(const EmbedBwdArgs& a, const RowParts& r, int from, int to, int step, int v, f2x (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = 0ull;
#pragma unroll 8
    for (int i = from; i < to; i += step) {
        const float4* p = reinterpret_cast<const float4*>(part_at(a, r, i, v));
        const float4 q0 = __ldcg(p), q1 = __ldcg(p + 1);
        s[0] = add2(s[0], pk2(q0.x, q0.y));
        s[1] = add2(s[1], pk2(q0.z, q0.w));
        s[2] = add2(s[2], pk2(q1.x, q1.y));
        s[3] = add2(s[3], pk2(q1.z, q1.w));
    }
}
// Counters of a chunk: 0 of a group of parts whose first is there and not the row's first, 1 of the first group of the row
// that begins there, 2 of that row's groups.  How many were done before.
__device__ __forceinline__ int done_here(const EmbedBwdArgs& a, int chunk, int which) {
    return atomicAdd(a.done + (3LL * chunk + which) * gridDim.y + blockIdx.y, 1);
}

// Sums of a chunk's rows (blockIdx.x < chunks) in columns blockIdx.y, 8 a thread; zeros for the rows without a token.
__global__ void __launch_bounds__(kSumThreads, 6) embedding_sum_kernel(const EmbedBwdArgs a, int rows, int chunks) {
    __shared__ int2 place[kEmbedChunk];
    __shared__ uint32_t empty;
    __shared__ int join[2];
    __shared__ bool last_group;
    pdl_trigger();
    pdl_wait();
    const int nv = a.D / 8, v = blockIdx.y * blockDim.x + threadIdx.x;
    if ((int)blockIdx.x >= chunks) {
        // 32 rows looked up at a time, then written
        const f2x none[4] = {0ull, 0ull, 0ull, 0ull};
        const int all = a.owners * rows, step = (gridDim.x - chunks) * 32, width = a.f32 ? 2 : 1;
        for (int s0 = (blockIdx.x - chunks) * 32; s0 < all; s0 += step) {
            if (threadIdx.x < 32) {
                const int s = s0 + threadIdx.x;
                const uint32_t m = __ballot_sync(0xffffffffu, s < all && __ldcg(a.first + min(s, all)) == __ldcg(a.first + min(s + 1, all)) &&
                                                                  vocabulary_row(a, rows, s) < a.V);
                if (threadIdx.x == 0) empty = m;
            }
            __syncthreads();
            if (v < nv)
                for (uint32_t m = empty; m != 0u; m &= m - 1u) {
                    uint4* p = static_cast<uint4*>(a.dw) + (vocabulary_row(a, rows, s0 + __ffs(m) - 1) * nv + v) * width;
                    if (a.f32)
                        put_pairs(reinterpret_cast<float*>(p), none);
                    else
                        *p = make_uint4(0u, 0u, 0u, 0u);
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
    const int head = place[0].y, tail = place[n - 1].y;
    const bool from = __ldcg(a.first + head) < i0, to = __ldcg(a.first + tail + 1) > i0 + n;
    f2x s[4] = {0ull, 0ull, 0ull, 0ull};
    constexpr int AHEAD = 4;
#pragma unroll 1
    for (int i = 0; i < n && v < nv; i += AHEAD) {
        uint4 q[AHEAD];
        Old old[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i + k >= n) continue;
            q[k] = __ldg(reinterpret_cast<const uint4*>(a.dy) + (long long)place[i + k].x * nv + v);
            if (a.accumulate && (i + k + 1 == n || place[i + k + 1].y != place[i + k].y))
                old[k] = old_row(a, vocabulary_row(a, rows, place[i + k].y), v);
        }
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
                put_pairs(a.part + (2LL * blockIdx.x) * a.D + 8 * v, s);
            else if (row == tail && to)
                put_pairs(a.part + (2LL * blockIdx.x + 1) * a.D + 8 * v, s);
            else
                put_row(a, vocabulary_row(a, rows, row), v, s, a.accumulate ? old[k] : Old{});
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = 0ull;
        }
    }
    if (!from && !to) return;
    // this CTA's parts are written: whether they were the last of their rows, or of a group of them
    __threadfence();
    __syncthreads();
    if (threadIdx.x < 2) {
        const int row = threadIdx.x == 0 ? head : tail;
        bool last = false;
        if (threadIdx.x == 0 ? from : to && !(from && head == tail)) {
            const RowParts r = parts_of(a, row);
            const int g = (blockIdx.x - r.first) / kJoin * kJoin;
            last = done_here(a, r.first + g, g == 0 ? 1 : 0) == min(kJoin, r.count - g) - 1;
        }
        join[threadIdx.x] = last ? row : -1;
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        const int row = join[w];
        if (row < 0) continue;
        const RowParts r = parts_of(a, row);
        const int g = (blockIdx.x - r.first) / kJoin * kJoin;
        const long long out = vocabulary_row(a, rows, row);
        Old old = {};   // (asked for ahead of the parts)
        __threadfence();
        if (r.count <= kJoin && v < nv) old = old_row(a, out, v);
        if (v < nv) add_parts(a, r, g, min(r.count, g + kJoin), 1, v, s);
        if (r.count > kJoin) {
            // the group's sum takes the place of its first part
            if (v < nv) put_pairs(part_at(a, r, g, v), s);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) last_group = done_here(a, r.first, 2) == (r.count - 1) / kJoin;
            __syncthreads();
            if (!last_group) continue;
            __threadfence();
            if (v < nv) {
                old = old_row(a, out, v);
                add_parts(a, r, 0, r.count, kJoin, v, s);
            }
        }
        if (v < nv) put_row(a, out, v, s, old);
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
long long embed_dones(long long T, int D) { return 3 * embed_chunks(T) * ((D / 8 + kSumThreads - 1) / kSumThreads); }
long long embed_chunks(long long T) { return (T + kEmbedChunk - 1) / kEmbedChunk; }

cudaError_t launch_embedding(const EmbedArgs& a, cudaStream_t s, bool pdl) {
    return a.w32 ? fwd_as<true>(a, s, pdl) : fwd_as<false>(a, s, pdl);
}
cudaError_t launch_embedding_sort(const EmbedBwdArgs& a, cudaStream_t s, bool pdl) {
    const int rows = owner_rows(a);
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(embedding_sort_kernel), kSortWarps * kSortRows * sizeof(int), allowed);
    if (e != cudaSuccess) return e;
    return launch_ex(embedding_sort_kernel, dim3((unsigned)a.owners), dim3(kSortWarps * 32), kSortWarps * rows * sizeof(int), s, pdl, a,
                     rows, (int)embed_dones(a.T, a.D));
}
cudaError_t launch_embedding_sum(const EmbedBwdArgs& a, cudaStream_t s, bool pdl) {
    const int rows = owner_rows(a), chunks = (int)embed_chunks(a.T), blocks = (a.D / 8 + kSumThreads - 1) / kSumThreads;
    const int zero = a.accumulate ? 0 : std::min((a.owners * rows + 31) / 32, 152 * 8);
    const int threads = std::min(kSumThreads, lanes_of(a.D));
    return launch_ex(embedding_sum_kernel, dim3((unsigned)(chunks + zero), (unsigned)blocks), dim3((unsigned)threads), 0, s, pdl, a,
                     rows, chunks);
}

}  // namespace lrs

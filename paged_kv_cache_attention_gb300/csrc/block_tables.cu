// block_tables.cu -- block tables, slots, positions and offsets of a step's tokens
// from the requests' lengths (the bookkeeping before a cache write: vLLM
// attention.py, InputMetadata's slot_mapping and block_tables; the placement of
// transformers docs "paged_attention", decode path).
//
// Request r goes from old to new tokens: have = ceil(old / bs), want = ceil(new /
// bs).  Released pages (entries want .. have - 1 of shrinking requests) are R in
// request order, taken ones (have .. want - 1) A.  The free pages are a stack of
// height F, the released ones on top of it with the first of them topmost:
//   page j that is taken = released[j]                 j < R
//                          free[F - 1 - (j - R)]       else
//   free[F + R - 1 - i]  = released[i]                 i >= A
// so one index i over max(A, R) says both what is read and where it goes: an
// entry has one reader, which also clears it, and reads and writes of the stack
// never meet.  Giving back the pages just taken restores the stack.
//
// A small step is bound by the launch and a chain of dependent loads (12 bytes per page
// moved, 16 per token), a large one by the eight SMs that do it: their issue slots are 52 %
// busy, with two binary searches for a page moved and one for a row, between barriers.  One
// cluster of eight CTAs, each with the prefix sums of all requests in its own shared
// memory, and cluster barriers between check, tables and rows, in place of a launch for
// each.  A step of at most kFew requests,
// pages and rows is the first CTA's alone (64 requests of a token each: 6.1 us, 7.4 with
// the cluster's barriers).  Rows beyond kRowsHere take a second launch over all SMs (near
// it both measure the same: 12K rows 8.4 us here, 8.2 there).
//
// Measured: 1000 requests of a token each 8.9 us, of 250 to 500 tokens 13.7 us (8.4 MB
// written for the two calls that its figure is the mean of: 0.6 us at HBM's rate).
#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kRowsHere = 16384;
constexpr int kRowThreads = 256;
constexpr int kAtOnce = 4;  // searches and loads that a thread has in flight
constexpr int kRowsPerCta = kRowThreads * kAtOnce;

// For each of i: the largest r in [0, n) with cu[r] <= i (cu[0] = 0 <= i), the request
// of item i.  step: the largest power of two below n (0 for n <= 1).
__device__ __forceinline__ void find(const int32_t *cu, int n, int step, const int (&i)[kAtOnce],
                                     int (&r)[kAtOnce]) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) r[k] = 0;
    for (; step > 0; step >>= 1)
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r[k] + step < n && cu[r[k] + step] <= i[k]) r[k] += step;
}

__device__ __forceinline__ int first_step(int n) { return n <= 1 ? 0 : 1 << (31 - __clz(n - 1)); }

// Slots and positions of rows t, t + stride, .. (kAtOnce of them); FRESH: table entries
// from L2, where another SM may just have written them.
template <bool FRESH>
__device__ __forceinline__ void write_rows(const TableParams &p, const int32_t *cu, int64_t t0,
                                           int stride, int total) {
    int t[kAtOnce], r[kAtOnce], x[kAtOnce], id[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) t[k] = (int)min(t0 + (int64_t)k * stride, (int64_t)p.rows);
    find(cu, p.batch, first_step(p.batch), t, r);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
        x[k] = t[k] < total ? __ldg(p.old_len + r[k]) + t[k] - cu[r[k]] : 0;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
        const int32_t *e = p.block_table + (int64_t)r[k] * p.max_blocks_per_seq + (x[k] >> p.bs_shift);
        id[k] = t[k] < total ? (FRESH ? __ldcg(e) : *e) : 0;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
        if (t[k] < p.rows) {
            p.slots[t[k]] = t[k] < total ? ((int64_t)id[k] << p.bs_shift) + (x[k] & (p.block_size - 1))
                                         : -1;
            p.positions[t[k]] = x[k];
        }
}

// Sums that stay at 2^32 - 1 (each is compared with a limit below that).
struct Sums {
    uint32_t tok, keys, taken, gone;
};

__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;
    return s < a ? 0xffffffffu : s;
}

__device__ __forceinline__ Sums add(const Sums &a, const Sums &b) {
    return {add_up(a.tok, b.tok), add_up(a.keys, b.keys), add_up(a.taken, b.taken),
            add_up(a.gone, b.gone)};
}

__device__ __forceinline__ Sums shift_up(const Sums &a, int d) {
    return {__shfl_up_sync(0xffffffffu, a.tok, d), __shfl_up_sync(0xffffffffu, a.keys, d),
            __shfl_up_sync(0xffffffffu, a.taken, d), __shfl_up_sync(0xffffffffu, a.gone, d)};
}

__device__ __forceinline__ Sums of_lane(const Sums &a, int l) {
    return {__shfl_sync(0xffffffffu, a.tok, l), __shfl_sync(0xffffffffu, a.keys, l),
            __shfl_sync(0xffffffffu, a.taken, l), __shfl_sync(0xffffffffu, a.gone, l)};
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(const TableParams p) {
    extern __shared__ int32_t s_cu[];  // [3][batch + 1]: rows, taken and released before r
    int32_t *s_tok = s_cu, *s_take = s_tok + p.batch + 1, *s_gone = s_take + p.batch + 1;
    __shared__ Sums s_warp[kThreads / 32];
    __shared__ uint32_t s_bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = (int)cluster_rank();
    const int B = p.batch, M = p.max_blocks_per_seq, shift = p.bs_shift;

    pdl_wait();
    if (threadIdx.x == 0) s_bad = 0;
    uint32_t bad = 0;
    const int F = *p.num_free;
    const long long cap = (long long)M << shift;
    Sums run = {0, 0, 0, 0};  // of the requests before this chunk
    for (int r0 = 0; r0 < B; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        Sums v = {0, 0, 0, 0};
        if (r < B) {
            int a = p.old_len[r], b = p.new_len[r];
            if (a < 0 || b < 0 || a > cap || b > cap) {
                bad |= PKV_DEVERR_SEQLEN;
                a = b = 0;
            }
            const int have = (a + p.block_size - 1) >> shift, want = (b + p.block_size - 1) >> shift;
            v.tok = (uint32_t)max(b - a, 0);
            v.keys = (uint32_t)b;
            v.taken = (uint32_t)max(want - have, 0);
            v.gone = (uint32_t)max(have - want, 0);
        }
        Sums in = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums o = shift_up(in, d);
            if (lane >= d) in = add(in, o);
        }
        if (lane == 31) s_warp[warp] = in;
        __syncthreads();
        static_assert(kThreads == 32 * 32, "a lane for each warp");
        const int used = min((B - r0 + 31) / 32, 32);  // warps that have a request
        Sums warps = s_warp[lane];  // up to and with warp `lane`
        for (int d = 1; d < used; d <<= 1) {
            const Sums o = shift_up(warps, d);
            if (lane >= d) warps = add(warps, o);
        }
        Sums before = add(run, in);  // up to and with r
        if (warp > 0) before = add(before, of_lane(warps, warp - 1));
        run = add(run, of_lane(warps, used - 1));
        if (r < B) {
            s_tok[r + 1] = (int)before.tok;
            s_take[r + 1] = (int)before.taken;
            s_gone[r + 1] = (int)before.gone;
            if (rank == 0) {
                p.cu_q[r + 1] = (int)before.tok;
                p.cu_k[r + 1] = (int)before.keys;
            }
        }
        __syncthreads();  // s_warp is used again
    }
    if (threadIdx.x == 0) {
        s_tok[0] = s_take[0] = s_gone[0] = 0;
        if (rank == 0) p.cu_q[0] = p.cu_k[0] = 0;
    }
    if (run.tok > (uint32_t)p.rows || run.keys > 0x7fffffffu) bad |= PKV_DEVERR_SEQLEN;
    // more pages than the pool has: an entry of the tables or the stack is there twice
    const int64_t height = F + (int64_t)run.gone - run.taken;
    if (F < 0 || F > p.num_blocks || run.gone > p.num_blocks || height > p.num_blocks)
        bad |= PKV_DEVERR_BLOCK_ID;
    if (height < 0) bad |= PKV_DEVERR_NO_BLOCKS;
    const int total = (int)run.tok, A = (int)run.taken, R = (int)run.gone;
    // A small step (all CTAs see the same sums) is done by the first CTA alone, without
    // the cluster's barriers.
    constexpr int kFew = kAtOnce * kThreads;
    const bool alone = max(run.taken, run.gone) <= (uint32_t)kFew && p.rows <= kFew && B <= kFew;
    if (alone && rank > 0) return;
    const int gtid = rank * kThreads + threadIdx.x, all = alone ? kThreads : kCluster * kThreads;
    auto sync = [&] {
        if (alone)
            __syncthreads();
        else
            cluster_sync();
    };
    const bool countable = __syncthreads_or((int)bad) == 0;

    const int moves = max(A, R), step = first_step(B);
    // The pages `all` apart from i on: ids, and the entries of the table that they leave
    // (nullptr: of the stack).
    auto pages_from = [&](int i, int (&id)[kAtOnce], int32_t *(&from)[kAtOnce]) {
        int at[kAtOnce], r[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) at[k] = min(i + k * all, moves);
        find(s_gone, B, step, at, r);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            from[k] = nullptr;
            if (at[k] < R) {
                const int want = (__ldg(p.new_len + r[k]) + p.block_size - 1) >> shift;
                from[k] = p.block_table + (int64_t)r[k] * M + want + (at[k] - s_gone[r[k]]);
            }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            id[k] = at[k] < R ? *from[k] : at[k] < moves ? p.free_blocks[F - 1 - (at[k] - R)] : 0;
    };
    int id[kAtOnce];
    int32_t *from[kAtOnce];
    if (countable) {
        // every id that will be moved, and the pages that new tokens go on filling
        for (int i = gtid; i < moves; i += kAtOnce * all) {
            pages_from(i, id, from);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (id[k] < 0 || id[k] >= p.num_blocks) bad |= PKV_DEVERR_BLOCK_ID;
        }
        for (int r = gtid; r < B; r += all) {
            const int a = p.old_len[r];
            if (p.new_len[r] > a && (a & (p.block_size - 1))) {
                const int e = p.block_table[(int64_t)r * M + (a >> shift)];
                if (e < 0 || e >= p.num_blocks) bad |= PKV_DEVERR_BLOCK_ID;
            }
        }
    }
    if (bad) atomicOr(&s_bad, bad);
    sync();  // every CTA has read num_free and checked its part
    bad = s_bad;
    if (!alone)
#pragma unroll
        for (int c = 0; c < kCluster; ++c) bad |= cluster_ld32(cluster_addr(smem_u32(&s_bad), c));
    if (bad) {  // nothing is moved, no row has a slot, no request a query or a key
        if (gtid == 0) flag_error(p.dev_error, bad);
        if (rank == 0)
            for (int r = threadIdx.x; r <= B; r += kThreads) p.cu_q[r] = p.cu_k[r] = 0;
        if (p.rows_here)
            for (int t = gtid; t < p.rows; t += all) {
                p.slots[t] = -1;
                p.positions[t] = 0;
            }
        sync();  // the others may still read s_bad
        return;
    }
    for (int i = gtid; i < moves; i += kAtOnce * all) {
        if (moves > kAtOnce * all) pages_from(i, id, from);  // (else: as they were checked)
        int at[kAtOnce], r[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) at[k] = min(i + k * all, moves);
        find(s_take, B, step, at, r);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (from[k]) *from[k] = -1;
            if (at[k] < A) {
                const int have = (__ldg(p.old_len + r[k]) + p.block_size - 1) >> shift;
                p.block_table[(int64_t)r[k] * M + have + (at[k] - s_take[r[k]])] = id[k];
            } else if (at[k] < moves) {
                p.free_blocks[F + R - 1 - at[k]] = id[k];
            }
        }
    }
    if (gtid == 0) *p.num_free = F + R - A;
    sync();  // the tables are written
    if (p.rows_here)
        for (int t = gtid; t < p.rows; t += kAtOnce * all)
            write_rows<true>(p, s_tok, t, all, total);
}

__global__ void __launch_bounds__(kRowThreads) block_rows_kernel(const TableParams p) {
    extern __shared__ int32_t s_cu[];
    pdl_wait();
    for (int r = threadIdx.x; r <= p.batch; r += kRowThreads) s_cu[r] = p.cu_q[r];
    __syncthreads();
    write_rows<false>(p, s_cu, (int64_t)blockIdx.x * kRowsPerCta + threadIdx.x, kRowThreads,
                      s_cu[p.batch]);
}

}  // namespace

cudaError_t launch_block_tables(const TableParams &p0, cudaStream_t stream) {
    TableParams p = p0;
    p.rows_here = p.rows <= kRowsHere;
    const int smem = 3 * (p.batch + 1) * 4;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(block_tables_kernel), smem);
    if (e != cudaSuccess) return e;
    e = launch_cluster(block_tables_kernel, kCluster, kCluster, kThreads, smem, stream, p);
    if (e != cudaSuccess || p.rows_here) return e;
    const int smem2 = (p.batch + 1) * 4;
    e = ensure_dynamic_smem(reinterpret_cast<const void *>(block_rows_kernel), smem2);
    if (e != cudaSuccess) return e;
    return launch_pdl(block_rows_kernel,
                      dim3((unsigned)((p.rows + (int64_t)kRowsPerCta - 1) / kRowsPerCta)),
                      dim3(kRowThreads), smem2, stream, p);
}

}  // namespace pkv

// step_tables.cu -- the tables of a decoding step, built on the device from
// the sequences' lengths: query offsets, new context lengths, block-table
// entries taken from a free list, the slot map, rotary positions and the
// visibility masks of drafted trees.
//
// With n_b new tokens on c_b committed rows, q_off is the exclusive prefix sum
// of n_b, and sequence b takes max(0, ceil((c_b + n_b) / P) - held_b) pages
// from the free list behind those of the sequences before it (a second
// prefix sum).  Only a CTA that has both sums can tell whether the whole step
// fits, before anything advances; up to 256 sequences every CTA forms them
// for itself and then writes its part of the rows (one launch, bound by latency:
// a step reads and writes some 20 KB), more are summed by one CTA, with the
// rows in a second launch, and so are the tables of more than 1,024 rows (32
// a tree at least) whose outputs take their inputs' place: the first CTA would
// advance what the others still have to read.  64 trees of 16: 3.7 us, in place
// 5.8; 256 of them 4.3 and 6.1; 257 to 512 of them 7.4-7.7 either way; 256
// prompts of up to 256 tokens 4.1; 512 prompts of 128 9.3 and 9.9.
// A row's page is looked up in the held part of the block table or, behind
// it, in the free list itself, so rows do not wait for the new entries.
//
// A tree's mask is built by pointer jumping, a warp per sequence with two
// nodes per lane: after round s a node's mask holds its nearest 2^s
// ancestors-or-self and its link points 2^s up, so log2 of the nodes, at most
// six rounds, do.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "tree.h"

namespace dsa {
namespace {

struct TablesArgs {
    int32_t B, total_q, max_q, max_ctx;
    int64_t stride;
    PagesDev pg;
    const int32_t *n_new, *ctx_old, *parent, *held_old, *free_pages, *free_range;
    int32_t *held, *free_out, *q_off, *ctx_len, *slots, *positions, *table;
    uint64_t* mask;
    int32_t *first_new, *held_kept;   // workspace: [B + 1] prefix of new pages, [B] pages held before
    int32_t* head;                    // workspace: the free list's head before
    int32_t* status;
};

struct SeqNeed {
    int32_t n, c, held, fresh;
    int code;
};

__device__ __forceinline__ SeqNeed seq_need(const TablesArgs& a, int b) {
    SeqNeed s{0, 0, 0, 0, DSA_OK};
    if (b >= a.B) return s;
    s.n = __ldg(a.n_new + b);
    s.c = a.ctx_old[b];              // may be an output too: no read-only path
    const int32_t most = (a.mask || a.parent) ? min(a.max_q, DSA_MAX_TREE) : a.max_q;
    if (s.n < 0 || s.n > most || s.c < 0 || (int64_t)s.c + s.n > a.max_ctx) {
        s.code = DSA_ERR_BAD_BATCH;
        s.n = 0;
        return s;
    }
    if (a.pg.table) {
        s.held = a.held_old[b];
        const int32_t need = (int32_t)(((int64_t)s.c + s.n + (1 << a.pg.shift) - 1) >> a.pg.shift);
        if (s.held < 0 || s.held > a.pg.max_pages) s.code = DSA_ERR_BAD_BATCH;
        else s.fresh = max(need - s.held, 0);    // need <= max_pages: c + n <= max_ctx
    }
    return s;
}

// The last b with start[b] <= v (start ascending from start[0] <= v).
__device__ __forceinline__ int find_seq(const int32_t* start, int B, int32_t v) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int32_t slot_of(const TablesArgs& a, int b, int32_t pos, int32_t head) {
    if (!a.pg.table) return (int32_t)(b * a.stride + pos);
    const int32_t p = pos >> a.pg.shift, held = a.held_kept[b];
    const int32_t page = p < held ? a.table[(int64_t)b * a.pg.max_pages + p]
                                  : __ldg(a.free_pages + head + a.first_new[b] + (p - held));
    if ((uint32_t)page >= (uint32_t)a.pg.pool_pages) {
        latch_status(a.status, DSA_ERR_BAD_INDEX);
        return -1;
    }
    return (page << a.pg.shift) + (pos & ((1 << a.pg.shift) - 1));
}

// The trees' rows, a warp per sequence, H nodes per lane (node lane + 32 h).
template <int H>
__device__ __forceinline__ void write_trees(const TablesArgs& a, int64_t me, int64_t threads, int32_t head) {
    const int lane = (int)(me & 31);
    const int rounds = 32 - __clz(max(a.max_q, 2) - 1);
    for (int64_t b = me >> 5; b < a.B; b += threads >> 5) {
        const int32_t q0 = a.q_off[b], n = a.q_off[b + 1] - q0, c = a.ctx_len[b] - n;
        int32_t up[H], slot[H];
        uint64_t m[H];
        // parents and pages are on their way together
#pragma unroll
        for (int h = 0; h < H; ++h) up[h] = lane + 32 * h < n ? __ldg(a.parent + q0 + lane + 32 * h) : -1;
#pragma unroll
        for (int h = 0; h < H; ++h) slot[h] = lane + 32 * h < n ? slot_of(a, (int)b, c + lane + 32 * h, head) : -1;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int32_t i = lane + 32 * h;
            if (up[h] < -1 || up[h] >= i) {
                if (i < n) latch_status(a.status, DSA_ERR_BAD_INDEX);
                up[h] = -1;
            }
            m[h] = 1ull << i;
        }
#pragma unroll 1
        for (int s = 0; s < rounds; ++s) {
            uint64_t m2[H];
            int32_t u2[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int from = up[h] & 31;
                m2[h] = __shfl_sync(0xffffffffu, m[0], from);
                u2[h] = __shfl_sync(0xffffffffu, up[0], from);
                if (H > 1) {
                    const uint64_t high = __shfl_sync(0xffffffffu, m[H - 1], from);
                    const int32_t uhigh = __shfl_sync(0xffffffffu, up[H - 1], from);
                    if (up[h] >= 32) m2[h] = high, u2[h] = uhigh;
                }
                if (up[h] < 0) m2[h] = 0u, u2[h] = -1;
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                m[h] |= m2[h];
                up[h] = u2[h];
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int32_t i = lane + 32 * h;
            if (i >= n) continue;
            a.slots[q0 + i] = slot[h];
            a.positions[q0 + i] = c + __popcll(m[h]) - 1;
            if (a.mask) a.mask[q0 + i] = m[h];
        }
    }
}

// Rows and new block-table entries, by thread `me` of `threads`.
__device__ void write_rows(const TablesArgs& a, int64_t me, int64_t threads) {
    const int32_t rows = a.q_off[a.B], head = a.pg.table ? *a.head : 0;
    const int64_t first_row = a.parent ? (int64_t)rows : 0;      // a tree's rows are written below
    for (int64_t r = first_row + me; r < a.total_q; r += threads) {
        if (r >= rows) {
            a.slots[r] = -1;
            a.positions[r] = -1;
            if (a.mask) a.mask[r] = 0u;
            continue;
        }
        const int b = find_seq(a.q_off, a.B, (int32_t)r);
        const int32_t i = (int32_t)r - a.q_off[b], n = a.q_off[b + 1] - a.q_off[b];
        const int32_t pos = a.ctx_len[b] - n + i;
        a.slots[r] = slot_of(a, b, pos, head);
        a.positions[r] = pos;
        if (a.mask) a.mask[r] = ~0ull >> (63 - i);
    }
    if (a.parent) {
        if (a.max_q <= 32) write_trees<1>(a, me, threads, head);
        else write_trees<2>(a, me, threads, head);
    }
    if (a.pg.table) {
        const int32_t fresh = a.first_new[a.B];
        for (int64_t e = me; e < fresh; e += threads) {
            const int b = find_seq(a.first_new, a.B, (int32_t)e);
            a.table[(int64_t)b * a.pg.max_pages + a.held_kept[b] + ((int32_t)e - a.first_new[b])] =
                __ldg(a.free_pages + head + e);
        }
    }
}

// NT threads: all of them walk the same few hundred instructions, so a small
// batch is faster with fewer (256 prompts: 6.4 us with 256, 8.2 with 1024).
// kRows (at most NT sequences): the CTAs also write the rows.  Each forms all
// sums for itself, the first writes them, and each writes its part of the
// rows; with more than one CTA no output may be an input.
template <int NT, bool kRows>
__global__ void __launch_bounds__(NT) step_lengths_kernel(const TablesArgs a) {
    constexpr int kWarps = NT / 32;
    // the tables again for this CTA's own rows, which would read them back
    // from L2 otherwise
    __shared__ int32_t s_off[kRows ? NT + 1 : 1], s_ctx[kRows ? NT : 1];
    __shared__ int32_t s_first[kRows ? NT + 1 : 1], s_held[kRows ? NT : 1], s_head;
    __shared__ int64_t s_n[kWarps], s_f[kWarps];
    __shared__ uint64_t s_both[kWarps];
    __shared__ int s_code;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    if (tid == 0) s_code = DSA_OK;
    int32_t head = 0, tail = 0;
    if (a.pg.table) {
        head = a.free_range[0];
        tail = a.free_range[1];
    }
    // pass 1: does the whole step fit?
    int64_t n_sum = 0, f_sum = 0;
    SeqNeed s{};
    int worst = DSA_OK;
    for (int b = tid; b < a.B; b += NT) {
        s = seq_need(a, b);
        n_sum += s.n;
        f_sum += s.fresh;
        worst = max(worst, s.code);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n_sum += __shfl_xor_sync(0xffffffffu, n_sum, o);
        f_sum += __shfl_xor_sync(0xffffffffu, f_sum, o);
    }
    if (lane == 0) {
        s_n[warp] = n_sum;
        s_f[warp] = f_sum;
    }
    __syncthreads();
    if (worst != DSA_OK) atomicMax(&s_code, worst);
    int64_t all_n = lane < kWarps ? s_n[lane] : 0, all_f = lane < kWarps ? s_f[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all_n += __shfl_xor_sync(0xffffffffu, all_n, o);
        all_f += __shfl_xor_sync(0xffffffffu, all_f, o);
    }
    __syncthreads();
    int code = s_code;
    if (code == DSA_OK && all_n > a.total_q) code = DSA_ERR_BAD_BATCH;
    if (code == DSA_OK && a.pg.table) {
        if (head < 0 || tail < head || tail > a.pg.pool_pages) code = DSA_ERR_BAD_BATCH;
        else if (all_f > tail - head) code = DSA_ERR_NO_PAGES;
    }
    const bool go = code == DSA_OK, first_cta = !kRows || blockIdx.x == 0;
    if (!go && tid == 0 && first_cta) latch_status(a.status, code);
    // pass 2: the prefix sums and what advances, NT sequences at a time; both
    // sums fit 32 bits now and share one scan
    uint64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        if (a.B > NT || b >= a.B) s = seq_need(a, b);
        if (!go) s.n = s.fresh = 0;
        const uint64_t mine = (uint64_t)(uint32_t)s.n | (uint64_t)(uint32_t)s.fresh << 32;
        uint64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s_both[warp] = incl;
        __syncthreads();
        uint64_t sums = lane < kWarps ? s_both[lane] : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t up = __shfl_up_sync(0xffffffffu, sums, o);
            if (lane >= o) sums += up;
        }
        const uint64_t lower = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
        const uint64_t before = base + (warp ? lower : 0u);
        base += __shfl_sync(0xffffffffu, sums, 31);
        if (b < a.B) {
            // the outputs may be the inputs' own arrays: an element is read
            // (above, or here for a refused step) before it is written
            const int32_t off = (int32_t)(uint32_t)(before + incl);
            const int32_t first = (int32_t)((before + incl - mine) >> 32);
            const int32_t ctx = (go ? s.c : a.ctx_old[b]) + s.n;
            const int32_t held = go || !a.pg.table ? s.held : a.held_old[b];
            if (first_cta) {
                a.q_off[b + 1] = off;
                a.ctx_len[b] = ctx;
            }
            if (a.pg.table && first_cta) {
                a.held_kept[b] = held;
                a.held[b] = held + s.fresh;
                a.first_new[b] = first;
            }
            if (kRows) {
                s_off[b + 1] = off;
                s_ctx[b] = ctx;
                s_held[b] = held;
                s_first[b] = first;
            }
        }
        __syncthreads();
    }
    const int32_t fresh = (int32_t)(base >> 32);
    if (tid == 0) {
        if (first_cta) a.q_off[0] = 0;
        if (a.pg.table && first_cta) {
            a.first_new[a.B] = fresh;
            *a.head = head;
            a.free_out[0] = head + fresh;
            a.free_out[1] = tail;
        }
        if (kRows) {
            s_off[0] = 0;
            s_head = head;
            s_first[a.B] = fresh;
        }
    }
    if (kRows) {
        __syncthreads();
        TablesArgs l = a;
        l.q_off = s_off;
        l.ctx_len = s_ctx;
        l.first_new = s_first;
        l.held_kept = s_held;
        l.head = &s_head;
        write_rows(l, (int64_t)blockIdx.x * NT + tid, (int64_t)gridDim.x * NT);
    }
}

__global__ void __launch_bounds__(256) step_rows_kernel(const TablesArgs a) {
    pdl_wait();
    write_rows(a, (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

}  // namespace

size_t step_tables_bytes(int32_t batch) { return sizeof(int32_t) * ((size_t)2 * batch + 2); }

cudaError_t launch_step_tables(const BatchDev& bd, const PagesDev& pg, const int32_t* n_new, const int32_t* ctx_old,
                               const int32_t* parent, const int32_t* held_old, int32_t* held,
                               const int32_t* free_pages, const int32_t* free_range, int32_t* free_out,
                               int32_t* slots, int32_t* positions, uint64_t* mask, int32_t* scratch, int32_t* status,
                               cudaStream_t stream) {
    TablesArgs a{};
    a.B = bd.B;
    a.total_q = bd.total_q;
    a.max_q = bd.max_q;
    a.max_ctx = bd.max_ctx;
    a.stride = bd.stride;
    a.pg = pg;
    a.n_new = n_new;
    a.ctx_old = ctx_old;
    a.parent = parent;
    a.held_old = held_old;
    a.held = held;
    a.free_pages = free_pages;
    a.free_range = free_range;
    a.free_out = free_out;
    a.q_off = const_cast<int32_t*>(bd.q_off);       // outputs of this call
    a.ctx_len = const_cast<int32_t*>(bd.ctx_len);
    a.slots = slots;
    a.positions = positions;
    a.mask = mask;
    a.table = const_cast<int32_t*>(pg.table);
    a.first_new = scratch;
    a.held_kept = scratch + bd.B + 1;
    a.head = scratch + 2 * (int64_t)bd.B + 1;
    a.status = status;
    // what the rows and entries can come to: the step's rows, and the pages
    // that sequences may take (all of max_ctx for a fresh prompt)
    const int64_t per_seq = pg.table ? std::min<int64_t>(pg.max_pages, ((int64_t)bd.max_q >> pg.shift) + 2) : 0;
    const int64_t items = std::max<int64_t>(std::max<int64_t>(bd.total_q, per_seq * bd.B), parent ? 32 * bd.B : 0);
    // One launch where every CTA can form the sums for itself (a second one
    // takes the host 2 us): up to 256 sequences, and no array that one CTA may
    // still have to read when the first has advanced it.
    cudaError_t e;
    const bool apart = ctx_old != a.ctx_len && (!pg.table || (held_old != held && free_range != free_out));
    if (bd.B <= 256 && (apart || items <= 1024)) {
        const int64_t ctas = apart ? std::min<int64_t>((items + 255) / 256, 2 * num_sms()) : 1;
        step_lengths_kernel<256, true><<<(unsigned)std::max<int64_t>(ctas, 1), 256, 0, stream>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess) count_launches(1);
        return e;
    }
    if (bd.B <= 256) step_lengths_kernel<256, false><<<1, 256, 0, stream>>>(a);
    else step_lengths_kernel<1024, false><<<1, 1024, 0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    count_launches(1);
    cudaLaunchConfig_t cfg = {};
    if (items == 0) return e;                        // no rows and no pages
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((items + 255) / 256, 8 * num_sms()));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, step_rows_kernel, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace dsa

// ninfer_kv_tables: block tables, slots and positions of a step's new tokens from
// the requests' lengths, in one launch.
//
// Two prefix sums over the requests (new tokens, pages to take) and one lookup
// a token. Latency bounds a decode step and the 16 bytes written a token a large
// admission, so every CTA recomputes the sums instead of waiting for another one:
// thread i of the block sums a contiguous run of requests, the block scans the
// threads' sums, and a token then finds its run by binary search among them in
// shared memory and its request by walking the run. Four neighbouring tokens share one
// search and go out in 16-byte stores (7.2 us one by one, 6.0 us so, which is what the
// host took to launch it, for 512 requests with 465,000 new tokens, 7.75 MB).
#include "decode.cuh"

namespace ninfer {
namespace {

constexpr int kThreads = 1024;

struct TablesParams {
    const int32_t *lengths, *fresh, *free_pages;
    int32_t *table;
    int64_t *slots;
    int32_t *positions, *rows, *offsets, *lengths_out, *counts, *status;
    uint64_t table_stride;
    uint32_t requests, run, table_pages, free_count, capacity, vectors;
    FastDiv page;
};

__device__ __forceinline__ int32_t clamp31(uint64_t v) { return v > 0x7fffffffull ? 0x7fffffff : (int32_t)v; }

struct Request {
    uint32_t length, fresh;     // tokens held, new ones (both < 2^31)
    uint32_t held, pages;       // pages held, pages to take
};

__device__ __forceinline__ Request request(const TablesParams &p, uint32_t i) {
    Request r;
    const int32_t l = p.lengths[i], n = p.fresh ? p.fresh[i] : 1;
    r.length = l > 0 ? l : 0;
    r.fresh = n > 0 ? n : 0;
    const uint32_t q = p.page.div(r.length);
    r.held = q + (q * p.page.d != r.length);
    const uint32_t end = r.length + r.fresh, qe = p.page.div(end);   // < 2^32
    r.pages = qe + (qe * p.page.d != end) - r.held;
    return r;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesParams p) {
    __shared__ uint64_t s_tokens[kThreads], s_pages[kThreads];      // sums before thread i's run
    __shared__ uint64_t s_warp[2][33];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const uint64_t first = (uint64_t)tid * p.run, last = min(first + p.run, (uint64_t)p.requests);
    uint64_t tokens = 0, pages = 0;
    int bad = 0;
    for (uint64_t i = first; i < last; ++i) {
        const Request r = request(p, (uint32_t)i);
        tokens += r.fresh;
        pages += r.pages;
        if (blockIdx.x == 0) {
            if (p.lengths[i] < 0 || (p.fresh && p.fresh[i] < 0) || r.length + r.fresh > 0x7fffffffu) bad |= NINFER_KV_BAD_LENGTH;
            if (r.fresh && r.held + r.pages > p.table_pages) bad |= NINFER_KV_ROW_TOO_SHORT;     // fresh pages among them or not
        }
    }
    uint64_t t = tokens, g = pages;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const uint64_t a = __shfl_up_sync(~0u, t, s), b = __shfl_up_sync(~0u, g, s);
        if (lane >= s) {
            t += a;
            g += b;
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = t;
        s_warp[1][warp] = g;
    }
    __syncthreads();
    if (warp < 2) {
        uint64_t w = s_warp[warp][lane];
        const uint64_t own = w;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const uint64_t a = __shfl_up_sync(~0u, w, s);
            if (lane >= s) w += a;
        }
        s_warp[warp][lane] = w - own;
        if (lane == 31) s_warp[warp][32] = w;
    }
    __syncthreads();
    t += s_warp[0][warp] - tokens;
    g += s_warp[1][warp] - pages;
    s_tokens[tid] = t;
    s_pages[tid] = g;
    const uint64_t total = s_warp[0][32], taken = s_warp[1][32];
    __syncthreads();

    // outputs by request: the runs are dealt out to the CTAs
    if (tid % gridDim.x == blockIdx.x) {
        uint64_t at = t, base = s_pages[tid];
        for (uint64_t i = first; i < last; ++i) {
            const Request r = request(p, (uint32_t)i);
            if (p.offsets) p.offsets[i] = clamp31(at);
            if (p.lengths_out) p.lengths_out[i] = clamp31((uint64_t)r.length + r.fresh);
            // pages whose first token is past the slots: entered here, since the loop over tokens ends with the slots
            // (lengths are whatever the buffer holds, up to 2^31 - 1 a request, and no loop may follow them that far)
            if (at + r.fresh > p.capacity) {
                const uint64_t skip = p.capacity > at ? r.length + (p.capacity - at) : r.length;
                const uint64_t end = min((uint64_t)r.held + r.pages, (uint64_t)p.table_pages);
                for (uint64_t pi = max((uint64_t)r.held, (skip + p.page.d - 1) / p.page.d); pi < end; ++pi) {
                    const uint64_t q = base + (pi - r.held);
                    p.table[i * p.table_stride + pi] = q < p.free_count ? p.free_pages[q] : -1;
                }
            }
            at += r.fresh;
            base += r.pages;
        }
    }
    if (blockIdx.x == 0) {
        if (tid == 0) {
            if (p.offsets) p.offsets[p.requests] = clamp31(total);
            if (p.counts) {
                p.counts[0] = clamp31(total);
                p.counts[1] = clamp31(taken);
            }
            if (taken > p.free_count) bad |= NINFER_KV_OUT_OF_PAGES;
            if (total > p.capacity) bad |= NINFER_KV_OUT_OF_SLOTS;
        }
        if (bad && p.status) atomicOr(p.status, bad);
    }

    // outputs by token, four neighbours a thread (of one request, mostly: one search); the first new
    // token of a fresh page also enters the page
    const uint64_t real = min(total, (uint64_t)p.capacity);
    for (uint64_t k0 = 4 * ((uint64_t)blockIdx.x * kThreads + tid); k0 < p.capacity; k0 += 4ull * gridDim.x * kThreads) {
        uint32_t lo = 0;                     // last thread whose run starts at or before k0
#pragma unroll
        for (uint32_t s = kThreads / 2; s; s >>= 1)
            if (s_tokens[lo + s] <= k0) lo += s;
        uint64_t at = s_tokens[lo], base = s_pages[lo];
        uint32_t i = lo * p.run;
        Request r = {};
        if (k0 < real) r = request(p, i);
        int64_t slot[4];
        int32_t position[4], row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t k = k0 + j;
            slot[j] = position[j] = row[j] = -1;
            if (k >= real) continue;
            while (k >= at + r.fresh) {      // ends: k < real
                at += r.fresh;
                base += r.pages;
                r = request(p, ++i);
            }
            const uint32_t pos = r.length + (uint32_t)(k - at), pi = p.page.div(pos), in = pos - pi * p.page.d;
            int32_t page = -1;
            if (pi < p.table_pages) {
                int32_t *entry = p.table + i * p.table_stride + pi;
                if (pi < r.held) page = *entry;
                else {
                    const uint64_t q = base + (pi - r.held);
                    if (q < p.free_count) page = p.free_pages[q];
                    if (in == 0) *entry = page;
                }
            }
            slot[j] = page < 0 ? -1 : (int64_t)page * p.page.d + in;
            position[j] = clamp31(pos);
            row[j] = (int32_t)i;
        }
        if (p.vectors && k0 + 4 <= p.capacity) {
            if (p.slots) {
                reinterpret_cast<longlong2 *>(p.slots + k0)[0] = make_longlong2(slot[0], slot[1]);
                reinterpret_cast<longlong2 *>(p.slots + k0)[1] = make_longlong2(slot[2], slot[3]);
            }
            if (p.positions) *reinterpret_cast<int4 *>(p.positions + k0) = make_int4(position[0], position[1], position[2], position[3]);
            if (p.rows) *reinterpret_cast<int4 *>(p.rows + k0) = make_int4(row[0], row[1], row[2], row[3]);
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k0 + j >= p.capacity) break;
            if (p.slots) p.slots[k0 + j] = slot[j];
            if (p.positions) p.positions[k0 + j] = position[j];
            if (p.rows) p.rows[k0 + j] = row[j];
        }
    }
}

// A contiguous buffer, and whether it shares memory with rows of `row` bytes, `stride` apart.
struct Buffer {
    const void *at;
    uint64_t bytes;
    bool meets(const void *rows, uint64_t count, uint64_t row, uint64_t stride) const {
        const uint64_t a = reinterpret_cast<uint64_t>(at), b = reinterpret_cast<uint64_t>(rows);
        if (!at || !rows || !bytes || !row || !count) return false;
        if (count == 1) stride = row;
        if (a + bytes <= b || a >= b + (count - 1) * stride + row) return false;
        if (a <= b) return true;
        const uint64_t in = (a - b) % stride;
        return in < row || in + bytes > stride;
    }
};

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_kv_tables(const int32_t *lengths, const int32_t *new_tokens, uint64_t requests,
                                uint64_t page_size, const int32_t *free_pages, uint64_t free_count,
                                int32_t *block_table, uint64_t table_pages, uint64_t table_stride, int64_t *slots,
                                int32_t *positions, int32_t *token_rows, uint64_t capacity, int32_t *offsets,
                                int32_t *lengths_out, int32_t *counts, int32_t *status, ninfer_stream stream) {
    if (!lengths || !block_table) return fail(NINFER_ERR_INVALID_ARGUMENT, "tables: NULL lengths or block_table");
    if (free_count && !free_pages) return fail(NINFER_ERR_INVALID_ARGUMENT, "tables: NULL free_pages with a count");
    const uint64_t most = 0x7fffffffull;
    if (!requests || !page_size || !table_pages || requests > most || page_size > most || table_pages > most ||
        capacity > most || free_count > most)
        return fail(NINFER_ERR_SHAPE, "tables: %llu requests, pages of %llu tokens, %llu pages a row (each 1 to 2^31 - 1; "
                    "capacity and free_count up to 2^31 - 1)", (unsigned long long)requests,
                    (unsigned long long)page_size, (unsigned long long)table_pages);
    if (table_stride < table_pages && requests > 1) return fail(NINFER_ERR_SHAPE, "tables: table_stride < table_pages");
    if (table_stride > (1ull << 40)) return fail(NINFER_ERR_OVERFLOW, "tables: table_stride over 2^40");
    for (const void *a : {(const void *)lengths, (const void *)new_tokens, (const void *)free_pages,
                          (const void *)block_table, (const void *)positions, (const void *)token_rows,
                          (const void *)offsets, (const void *)lengths_out, (const void *)counts, (const void *)status})
        if (!aligned(a, 4)) return fail(NINFER_ERR_ALIGNMENT, "tables: int32 buffers must be 4-byte aligned");
    if (!aligned(slots, 8)) return fail(NINFER_ERR_ALIGNMENT, "tables: slots must be 8-byte aligned");
    // every CTA reads the inputs while others write (the row of a table that another one fills is not read)
    const Buffer in[] = {{lengths, 4 * requests}, {new_tokens, 4 * requests}, {free_pages, 4 * free_count}};
    const Buffer outs[] = {{slots, 8 * capacity}, {positions, 4 * capacity}, {token_rows, 4 * capacity}, {offsets, 4 * (requests + 1)},
                           {lengths_out, 4 * requests}, {counts, 8}, {status, 4}};
    for (const Buffer &i : in) {
        bool shared = i.meets(block_table, requests, 4 * table_pages, 4 * table_stride);
        for (const Buffer &o : outs) shared |= o.meets(i.at, 1, i.bytes, i.bytes);
        if (shared) return fail(NINFER_ERR_INVALID_ARGUMENT, "tables: an output overlaps an input (lengths_out may not be lengths)");
    }
    for (const Buffer &o : outs)
        if (o.meets(block_table, requests, 4 * table_pages, 4 * table_stride))
            return fail(NINFER_ERR_INVALID_ARGUMENT, "tables: an output overlaps block_table");
    TablesParams p;
    p.lengths = lengths;
    p.fresh = new_tokens;
    p.free_pages = free_pages;
    p.table = block_table;
    p.slots = slots;
    p.positions = positions;
    p.rows = token_rows;
    p.offsets = offsets;
    p.lengths_out = lengths_out;
    p.counts = counts;
    p.status = status;
    p.table_stride = table_stride;
    p.requests = (uint32_t)requests;
    p.run = (uint32_t)((requests + kThreads - 1) / kThreads);
    p.table_pages = (uint32_t)table_pages;
    p.free_count = (uint32_t)free_count;
    p.capacity = (uint32_t)capacity;
    p.vectors = aligned(slots, 16) && aligned(positions, 16) && aligned(token_rows, 16);
    p.page = FastDiv((uint32_t)page_size);
    const uint64_t work = capacity / 4 > requests ? capacity / 4 : requests;
    const uint64_t want = (work + kThreads - 1) / kThreads;
    return launch_dependent("tables", tables_kernel, dim3((unsigned)(want < 304 ? want : 304)), dim3(kThreads), 0,
                            (cudaStream_t)stream, p);
}

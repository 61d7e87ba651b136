// fa_cache.cu -- the paged key/value cache's bookkeeping: fa_page_plan (block
// tables and slot maps from request lengths) and fa_kv_store (rows into pages).
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kPlanMaxB = kMaxVarlenSeqs;   // one thread per request in the scans

struct PlanArgs {
    const int* ctx;
    const int* fresh;
    int* table;
    int* ring;
    const long long* pool;
    long long* pool_out;
    int* cu;
    int* kv;
    int* slots;
    int B, W, P, num_slots, ps_log2;
};

// Inclusive scan over the block of (tokens, pages in, pages out), one request
// a thread; the tokens in 64 bits, since nothing bounds their sum.
struct Scan3 {
    long long n;
    int in, out;
};

__device__ __forceinline__ Scan3 warp_scan(Scan3 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long n = __shfl_up_sync(0xffffffffu, v.n, o);
        const int in = __shfl_up_sync(0xffffffffu, v.in, o), out = __shfl_up_sync(0xffffffffu, v.out, o);
        if (lane >= o) {
            v.n += n;
            v.in += in;
            v.out += out;
        }
    }
    return v;
}

// Index of the request whose range [pref[b], pref[b + 1]) holds x (x < pref[B]).
__device__ __forceinline__ int find_request(const int* pref, int B, int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (pref[mid + 1] > x) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// Every block scans all requests (their lengths are a few KB) and then takes
// its share of the slots, of the pages handed out and of the pages taken back;
// the three lists are flat, so a few long prompts and a thousand single tokens
// spread alike.  A token's page is read from where it comes from (the table
// for a page that the request had, the ring for a new one), so no block waits
// for another's table entries and one launch does it all.
//   have = ceil(c / page), need = min(ceil((c + n) / page), W),
//   slot of position x = entry[x / page] * page + x % page.
// Bound by latency: lengths, scan, search and page lookup depend on one another.
// From cold caches 5 us on the GPU for 8 requests, 8.5 for 1000 (the scan over 32
// warps), 7.9 for 560000 rows of 128 prompts (2.2 MB; the first block's count of
// the pages is the last to end).  Calls from Python one behind the other 7.3 to
// 8.8 us, replays of a graph of one call 6.2, 8.5 and 8.3.
__global__ void __launch_bounds__(1024) page_plan_kernel(const PlanArgs a) {
    __shared__ int s_cu[kPlanMaxB + 1], s_in[kPlanMaxB + 1], s_out[kPlanMaxB + 1];
    __shared__ int s_ctx[kPlanMaxB];
    __shared__ Scan3 s_warp[32];
    __shared__ long long s_lost[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    grid_launch_next();
    grid_wait();
    const int W = a.W, P = a.P, sh = a.ps_log2;
    const long long cap = (long long)W << sh, up = (1 << sh) - 1;

    long long head = a.pool[0], free_n = 0;
    head = head < 0 ? 0 : head;
    free_n = a.pool[1] - head;
    free_n = free_n < 0 ? 0 : (free_n > P ? P : free_n);
    const int avail = (int)free_n, room = P - avail, head_p = (int)(head % P);
    const int tail_p = head_p + avail >= P ? head_p + avail - P : head_p + avail;

    Scan3 v = {0, 0, 0};
    long long lost = 0;
    int have = 0;
    if (tid < a.B) {
        long long c = a.ctx[tid];
        c = c < 0 ? 0 : (c > cap ? cap : c);
        const int f = a.fresh[tid];
        have = (int)((c + up) >> sh);
        s_ctx[tid] = (int)c;
        if (f < 0) {
            v.out = have;
            if (blockIdx.x == 0) a.kv[tid] = 0;
        } else {
            const long long total = c + f, every = (total + up) >> sh, need = every < W ? every : W;
            v.n = f;
            v.in = (int)need - have;
            lost = every - need;
            if (blockIdx.x == 0) a.kv[tid] = (int)(total < cap ? total : cap);
        }
    }
    v = warp_scan(v, lane);
#pragma unroll
    for (int o = 16; o; o >>= 1) lost += __shfl_down_sync(0xffffffffu, lost, o);
    if (lane == 31) s_warp[warp] = v;
    if (lane == 0) s_lost[warp] = lost;
    __syncthreads();
    Scan3 before = {0, 0, 0};
    for (int w = 0; w < warp; ++w) {
        before.n += s_warp[w].n;
        before.in += s_warp[w].in;
        before.out += s_warp[w].out;
    }
    if (tid < a.B) {
        const long long n = before.n + v.n;
        s_cu[tid + 1] = n > 0x7fffffffLL ? 0x7fffffff : (int)n;
        s_in[tid + 1] = before.in + v.in;
        s_out[tid + 1] = before.out + v.out;
    }
    if (tid == 0) s_cu[0] = s_in[0] = s_out[0] = 0;
    __syncthreads();

    const int total_in = s_in[a.B], total_out = s_out[a.B];
    auto ring_at = [&](int idx) -> int {   // the idx-th free page, idx < avail <= P; -1: what is there is no page
        const int at = head_p + idx >= P ? head_p + idx - P : head_p + idx, page = a.ring[at];
        return page >= 0 && page < P ? page : -1;
    };
    if (blockIdx.x == 0) {
        // The first block sums up: offsets, the queue's counters, and the entries
        // handed out that are no pages (a request left with them in its row; they
        // serve no token, so they are missing as well).  Nothing else, since it
        // looks at all of the entries: with 9000 of them, and 560000 rows in the
        // other blocks, a call takes 8.4 us (11.4 with a share of the rows besides).
        for (int i = tid; i <= a.B; i += blockDim.x) a.cu[i] = s_cu[i];
        const int used = total_in < avail ? total_in : avail;
        int holes = 0;
        for (int i = tid; i < used; i += 8 * blockDim.x) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const long long x = i + (long long)e * blockDim.x;
                holes += x < used && ring_at((int)x) < 0;
            }
        }
        holes = __reduce_add_sync(0xffffffffu, holes);
        if (lane == 0) s_lost[warp] += holes;
        __syncthreads();
        if (tid == 0) {
            long long l = total_in - used;
            for (int w = 0; w < nw; ++w) l += s_lost[w];
            a.pool_out[0] = head + used;
            a.pool_out[1] = head + avail + (total_out < room ? total_out : room);
            a.pool_out[2] = l;
        }
        return;
    }
    const int stride = (gridDim.x - 1) * blockDim.x, first = (blockIdx.x - 1) * blockDim.x + tid;
    // Slots.  A row a thread while there are threads enough (single tokens: each
    // row is another request, and its lookups should not queue behind others');
    // else four rows at a time: one search, then requests and pages as they come
    // (a page is looked up once for the rows that lie in it).  Measured for 560000
    // rows of 128 prompts: 12.5 us a row at a time, 8 by fours; for 1000 single
    // tokens 10.4 us a row at a time, 12.9 by fours.
    const int per = a.num_slots <= stride ? 1 : 4;
    const bool wide = per == 4 && (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0;
    const int rows = s_cu[a.B];
    for (long long t0 = (long long)per * first; t0 < a.num_slots; t0 += (long long)per * stride) {
        int out[4] = {-1, -1, -1, -1};
        if (t0 < rows) {
            int b = find_request(s_cu, a.B, (int)t0), page = -1;
            long long at = -1;      // the column (of request b) that `page` is
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = (int)t0 + e;
                if (e >= per || t >= rows) continue;
                while (t >= s_cu[b + 1]) {
                    ++b;
                    at = -1;
                }
                const long long pos = (long long)s_ctx[b] + (t - s_cu[b]), col = pos >> sh;
                if (col >= W) continue;
                if (col != at) {
                    at = col;
                    const int hb = (int)(((long long)s_ctx[b] + up) >> sh);
                    if (col < hb) {
                        page = a.table[(long long)b * W + col];
                        if (page >= P) page = -1;
                    } else {
                        const int idx = s_in[b] + (int)col - hb;
                        page = idx < avail ? ring_at(idx) : -1;
                    }
                }
                if (page >= 0) out[e] = (page << sh) + (int)(pos & up);
            }
        }
        if (wide && t0 + 4 <= a.num_slots) {
            *reinterpret_cast<int4*>(a.slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < per && t0 + e < a.num_slots) a.slots[t0 + e] = out[e];
        }
    }
    // Pages handed out.
    for (long long i = first; i < total_in; i += stride) {
        const int b = find_request(s_in, a.B, (int)i);
        const int col = (int)(((long long)s_ctx[b] + up) >> sh) + (int)i - s_in[b];
        a.table[(long long)b * W + col] = i < avail ? ring_at((int)i) : -1;
    }
    // Pages taken back, behind the free ones.
    const int back = total_out < room ? total_out : room;
    for (long long i = first; i < back; i += stride) {
        const int b = find_request(s_out, a.B, (int)i);
        const int at = tail_p + i >= P ? (int)(tail_p + i - P) : (int)(tail_p + i);
        a.ring[at] = a.table[(long long)b * W + ((int)i - s_out[b])];
    }
}

struct StoreArgs {
    const uint4* k;
    const uint4* v;
    uint4* kp;
    uint4* vp;
    const int* slots;
    long long k_stride, v_stride;   // 16-byte chunks between tokens
    long long n;                    // chunks of all tokens
    int chunks, dlog, Hkv, ps_log2; // chunks a token, log2(chunks a row)
    long long num_slots;
};

// One 16-byte chunk of K and of V a thread and step; a token's row is read in
// the order of memory, and a head's row of a slot is a whole 128 bytes or more of
// the cache, so both sides move in full lines.  Bound by HBM: 328 MB (40000 rows
// of 8 heads of 128) in 47.5 us, 6.9 TB/s read and written together (a plain
// copy: 6.8).  64 rows: 4 us on the GPU, launch and three loads in a row (the slot,
// K's chunk, and V's, which does not move above the store of K's).  41 MB: 8.2.
__global__ void __launch_bounds__(256) kv_store_kernel(const StoreArgs a) {
    grid_launch_next();
    grid_wait();
    const long long stride = (long long)gridDim.x * blockDim.x;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < a.n; i += stride) {
        const long long t = i / a.chunks;
        const int c = (int)(i - t * a.chunks), h = c >> a.dlog, x = c & ((1 << a.dlog) - 1);
        const long long slot = a.slots[t];
        if (slot < 0 || slot >= a.num_slots) continue;
        const long long row = (((slot >> a.ps_log2) * a.Hkv + h) << a.ps_log2) + (slot & ((1 << a.ps_log2) - 1));
        const long long to = (row << a.dlog) + x;
        a.kp[to] = a.k[t * a.k_stride + c];
        a.vp[to] = a.v[t * a.v_stride + c];
    }
}

}  // namespace

int page_log2(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

}  // namespace fa

using namespace fa;

static bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

extern "C" {

int fa_page_plan(const int* ctx_lens, const int* new_lens, int B, int page_size, int* block_table, int table_width,
                 int* ring, int num_pages, const int64_t* pool, int64_t* pool_out, int* cu_new, int* kv_lens,
                 int* slots, int num_slots, cudaStream_t stream) {
    if (!ctx_lens || !new_lens || !block_table || !ring || !pool || !pool_out || !cu_new || !kv_lens)
        return FA_ERR_INVALID;
    if (B < 1 || table_width < 1 || num_pages < 1 || num_slots < 0 || (num_slots > 0 && !slots)) return FA_ERR_INVALID;
    const int lg = page_log2(page_size);
    if (lg < 0 || B > kPlanMaxB) return FA_ERR_UNSUPPORTED;
    if ((long long)B * table_width > 0x7fffffffLL || (long long)table_width * page_size > 0x7fffffffLL ||
        (long long)num_pages * page_size > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    if (misaligned(ctx_lens, 3) || misaligned(new_lens, 3) || misaligned(block_table, 3) || misaligned(ring, 3) ||
        misaligned(pool, 7) || misaligned(pool_out, 7) || misaligned(cu_new, 3) || misaligned(kv_lens, 3) ||
        misaligned(slots, 3))
        return FA_ERR_ALIGN;
    // Every block reads all lengths while others write: an output over any other
    // array (kv_lens over ctx_lens, say) would be a race.  The first three are
    // read only.
    const size_t n = B;
    const Span arrays[] = {{ctx_lens, 4 * n}, {new_lens, 4 * n}, {pool, 24}, {pool_out, 24}, {block_table, 4 * n * table_width},
                           {ring, 4 * (size_t)num_pages}, {cu_new, 4 * (n + 1)}, {kv_lens, 4 * n}, {slots, 4 * (size_t)num_slots}};
    for (int i = 3; i < 9; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(arrays[i], arrays[j])) return FA_ERR_INVALID;
    DevStatus* status = device_status_ptr();
    const int sms = fa_num_sms();
    if (!status || sms < 1) return FA_ERR_LAUNCH;
    PlanArgs a;
    a.ctx = ctx_lens;
    a.fresh = new_lens;
    a.table = block_table;
    a.ring = ring;
    a.pool = reinterpret_cast<const long long*>(pool);
    a.pool_out = reinterpret_cast<long long*>(pool_out);
    a.cu = cu_new;
    a.kv = kv_lens;
    a.slots = slots;
    a.B = B;
    a.W = table_width;
    a.P = num_pages;
    a.num_slots = num_slots;
    a.ps_log2 = lg;
    const int threads = B <= 256 ? 256 : (B + 31) / 32 * 32;
    // Blocks: one that sums up, and for the rest a slot a thread, four past a block
    // an SM, or 32 entries of the table that pages may go to or come from; at most
    // what the SMs hold at a time, since every block scans all requests first.
    const int each = num_slots <= sms * threads ? threads : 4 * threads;
    long long grid = ((long long)num_slots + each - 1) / each;
    const long long pages = ((long long)B * table_width + 32LL * threads - 1) / (32LL * threads), most = sms * (2048LL / threads);
    grid = grid > pages ? grid : pages;
    grid = 1 + (grid < 1 ? 1 : (grid > most - 1 ? most - 1 : grid));
    return launch_dependent(page_plan_kernel, (int)grid, threads, 0, stream, a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_kv_store(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int* slots, int T, int Hkv,
                int d, void* k_pages, void* v_pages, int num_pages, int page_size, cudaStream_t stream) {
    if (!k || !v || !slots || !k_pages || !v_pages) return FA_ERR_INVALID;
    if (T < 0 || Hkv < 1 || num_pages < 1 || d < 1) return FA_ERR_INVALID;
    const int lg = page_log2(page_size);
    if ((d != 64 && d != 128 && d != 256) || lg < 0) return FA_ERR_UNSUPPORTED;
    if (k_stride < (long long)Hkv * d || v_stride < (long long)Hkv * d) return FA_ERR_INVALID;
    if ((long long)Hkv * d > 0x7fffffffLL || (long long)num_pages * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    if (misaligned(k, 15) || misaligned(v, 15) || misaligned(k_pages, 15) || misaligned(v_pages, 15) ||
        misaligned(slots, 3) || (k_stride & 7) || (v_stride & 7))
        return FA_ERR_ALIGN;
    if (T == 0) return FA_OK;
    // One array for keys and values (a cache that keeps one row for both) can only
    // take the same rows for both; else two threads would write each slot.
    const size_t cache = (size_t)num_pages * Hkv * page_size * d * 2;
    if (overlap({k_pages, cache}, {v_pages, cache}) && !(k_pages == v_pages && k == v && k_stride == v_stride)) return FA_ERR_INVALID;
    if (overlap({slots, 4 * (size_t)T}, {k_pages, cache}) || overlap({slots, 4 * (size_t)T}, {v_pages, cache})) return FA_ERR_INVALID;
    const int sms = fa_num_sms();
    if (sms < 1) return FA_ERR_LAUNCH;
    StoreArgs a;
    a.k = static_cast<const uint4*>(k);
    a.v = static_cast<const uint4*>(v);
    a.kp = static_cast<uint4*>(k_pages);
    a.vp = static_cast<uint4*>(v_pages);
    a.slots = slots;
    a.k_stride = k_stride / 8;
    a.v_stride = v_stride / 8;
    a.dlog = d == 64 ? 3 : d == 128 ? 4 : 5;
    a.chunks = Hkv << a.dlog;
    a.n = (long long)T * a.chunks;
    a.Hkv = Hkv;
    a.ps_log2 = lg;
    a.num_slots = (long long)num_pages * page_size;
    long long grid = (a.n + 255) / 256;
    if (grid > 8LL * sms) grid = 8LL * sms;
    return launch_dependent(kv_store_kernel, (int)grid, 256, 0, stream, a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"

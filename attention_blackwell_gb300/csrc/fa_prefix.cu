// fa_prefix.cu -- fa_prefix_fwd: attention of new tokens over a shared prefix
// and each request's own paged keys (sm_103a, tcgen05 / TMEM / TMA).
//
// With x_j = alpha q . k_j over the keys that a row sees (the prefix's, then
// its request's own up to the causal limit), any split of the keys into sets s
// gives (m_s, l_s, O_s) = (max x, sum 2^(x - m_s), sum 2^(x - m_s) v), and
//   O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s,  M = max m_s.
// So the prefix's K and V are read once for a block of up to 256 query rows
// (the G query heads of a key/value head, times as many tokens of any requests
// as fit), a request's own once for the rows of its own tokens.  Both are the
// same work on different pages, so one persistent kernel does both:
//
//   item     one row block of one key/value head against one list of pages:
//            the prefix's (rows of any requests) or a request's (its rows);
//   unit     one tile of kN keys of one item;
//   worker   a contiguous range of the flat list of units, so the tiles, not
//            the requests, are shared out evenly whatever the lengths are; an
//            item cut by a range's end is a segment in each of its workers;
//   segment  leaves its rows' (m, l, O) (maximum, sum, unnormalised output) in
//            the workspace; segment ids are item + worker, unique because every
//            step along the list raises one of the two.
//
// A second kernel joins each output row's segments in fp32, in the list's order,
// so the result does not depend on timing.  A request with rows for four row
// blocks or more (a long prompt) gains nothing from sharing the prefix's tiles
// with other requests' rows: its items take the prefix's tiles and then their
// own, and one that no range cuts writes its output itself (six prompts of up to
// 2048 tokens over 8192 shared keys: 1226 us joined, 1113 so; from one row block
// up, batches that mix prompts and steps are up to 30 % slower).
//
// Some CTAs work on the prefix, the others on the requests, in proportion to
// the cost of both.  Within a CTA (d = 64 and 128), by the rows that a block of
// the prefix (all of the call's) or of a request (of max_seqlen tokens: one shape
// for all requests of a call) may have:
//   rows > 128    the CTA is one worker: two row tiles share every K/V tile (the
//                 ping-pong of fa_fwd.cu): the shape for the prefix of a large
//                 batch and for prompts, where the tensor core sets the pace;
//   rows <= 128   two workers, one for each softmax warpgroup, that share the
//                 loader, the ring of K/V tiles and the issuer, which serves
//                 them by turns;
//   rows <= 32    no tcgen05: every warp (or pair of warps) is a worker of its
//                 own (few_rows below): single tokens, where the copies set the
//                 pace.
// d = 256: one worker a CTA, one row tile, S double-buffered, 64-key tiles (its
// accumulator takes half of tensor memory), Q in tensor memory too, S and P V
// issued by a warp each; few rows only for requests of few keys (see few_items).
//
// Warps: softmax (8; at d = 256 four of them bring Q), loader, issuer (d = 256:
// two), and one or two that walk the list ahead of the others and leave each
// tile's description, page numbers included, in shared memory, so that no role
// waits for a table entry.
//
// Keys behind the end of a list and keys of absent pages are masked by
// selection, and their V rows are zeroed in shared memory before the product
// (0 * NaN would poison the sum), so the cache's leftovers never matter.
//
// What bounds it (GB300; 6.78 TB/s and 1892 TFLOP/s measured), 32 / 8 heads of
// 128 unless said otherwise:
//   64 single tokens, 8192 shared keys and a thousand own ones each (282 MB): 66
//   us, 57 in the main kernel.  HBM: 5.9 TB/s once every warp's ring is full,
//   which takes the first 12000 cycles (6 us: tables, walk, page numbers and first
//   copies depend on one another, on cold code); the join 8.
//   512 over 32768 (1.18 GB, 279 GFLOP): 343 to 349 us.  The prefix's CTAs take 3400
//   cycles a unit of two row tiles by 128 keys, 2048 of them products: each row
//   tile's chain S, softmax (1500), P V has one other's products to hide behind.
//   prompts, six of up to 2048 tokens over 8192 (1.43 TFLOP): 1070 to 1114 us,
//   tensor pipe 58 % busy in the main kernel, the same chain.
//   d = 256, one key/value head, 100 tokens over 16384 and 2000 own keys (224 MB,
//   60 GFLOP): 81 us; 1570 cycles a 64-key tile, 1024 of them products.
//   one request, one token: 15 to 17 us a call, the call from Python 13, the two
//   kernels 12.5 and 7 from cold caches, a graph of them 18.  With a table of 8192
//   pages, where the grid is all SMs, 2 more.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr float kTau = 8.0f;        // rescale threshold (log2 units), as in the forward kernels

constexpr int kMaxKeys = 1 << 29;   // of the prefix, of a request
constexpr int kFew = 0, kOne = 1, kTwo = 2;   // row tiles: 16 or 32 rows, 128, 2 x 128
constexpr int few_limit(int d) { return d == 256 ? 16 : 32; }   // rows up to which kFew is taken

template <int D> struct Pf {
    static constexpr int kStreams = D == 256 ? 1 : 2;
    static constexpr int kN = D == 256 ? 64 : 128;               // keys a tile
    static constexpr int kBoxes = D / 64;                        // 64-column boxes a row
    static constexpr uint32_t kKVBox = kN * 128u;                // bytes of a box of a K/V tile
    static constexpr uint32_t kTile = kBoxes * kKVBox;
    static constexpr uint32_t kQBox = 16384u;                    // 128 rows x 128 B
    static constexpr uint32_t kQTile = D == 256 ? 0 : kBoxes * kQBox;   // d = 256: Q is in tensor memory
    static constexpr int kLook = 3 - kStreams;                   // tiles of one worker with S in flight
    static constexpr int kRing = D == 64 ? 8 : D == 128 ? 4 : 6; // K/V tiles: 128 KB, at d = 256 192
    static constexpr uint32_t kTiles = 196608;                       // of them, or of the few rows' rings
    static constexpr int kThreads = 384;
    static constexpr int kMaxSmem = 232448 - 4096;               // dynamic; the rest is PfShared
    static_assert(kStreams * kQTile + kRing * kTile <= kTiles, "Q and the ring");
    static constexpr int kFewParts = 256 / D;               // few rows: 16-key parts a step, slots of a step's K or V a warp
    static constexpr uint32_t kFewRing = kTiles / 8 / (D * 32 * kFewParts);
    // Cycles a CTA takes for a unit of the prefix and of the requests' own keys,
    // by which the CTAs are divided between the two: measured in the kernel on
    // GB300, few rows with a third of the CTAs on the requests (512 single tokens
    // over 32768 keys: 50 of 152).  Where every CTA streams keys, HBM makes it 780,
    // 1520 and 2850 (d = 64, 128, 256; 6.6 to 7.2 TB/s read).  At d = 256, 900 is a
    // compromise: of nine batches, 1400 makes some 26 % faster and others 26 %
    // slower, 1875 (a warp's 15000, see few_items) 18 % and 34 %.
    // kTwo on the prefix: when several row blocks share a tile, L2 serves all but the
    // first; alone, each tile comes from HBM for 256 rows only, and its latency grows
    // with the share of the traffic (`own`, 0 to 1) that the requests' CTAs ask for at
    // the same time.
    __host__ __device__ static constexpr int few_cost(int halves) { return (D == 64 ? 520 : D == 128 ? 780 : 900) * halves; }
    // Few rows at d = 256, where each of eight warps takes 15000 cycles for a unit of
    // its own: worth it for items of few units (over_s of them for the item itself),
    // else one row tile.  100 keys a request of 8 heads: 44 us for 128 requests, one
    // row tile 60; 2000 keys and 16 requests over a long prefix: 107, one row tile 84.
    __host__ __device__ static constexpr bool few_items(int units, int items) { return D != 256 || units < 14LL * items; }
    __device__ static float cost_p(int mode, int halves, bool shared, float own) {
        return mode == kFew ? few_cost(halves) : mode == kOne ? (D == 64 ? 3800 : D == 128 ? 5000 : 1600)
             : D == 64 ? (shared ? 3400 : 3400 + 2600 * own) : (shared ? 3700 : 4400 + 4000 * own);
    }
    __device__ static float cost_s(int mode, int halves) {
        return mode == kFew ? few_cost(halves) : mode == kOne ? (D == 64 ? 3800 : D == 128 ? 5000 : 1550) : (D == 64 ? 3500 : 4000);
    }
    static constexpr uint32_t kColO1 = 128, kColS = 256, kColSStep = kN;   // O of the second worker or tile, S
    static constexpr uint32_t kColQ = 384;   // d = 256: Q, bf16 pairs
};

// Of a row of q, for the joining kernel: its request's first row, rows and keys
// (n = 0: no request), the units and items before it.
struct PfRow {
    int c0, n, s, pref, items, block, pad[2];   // block: its row block among the prefix's (index), -1: none
};
// The list of units, in shared memory.
struct PfTables {
    int* pref;           // [B+1] units of requests before b (all key/value heads)
    int* items;          // [B+1] items of requests before b
    int* cu;             // [B+1] sanitised offsets
    int* len;            // [B] own keys
    int* block;          // the prefix's row blocks, in units of tb rows of q (h.blocks of them; null: all)
};

// How the list is divided: the same in every CTA, left for the joining kernel.
struct PfHeader {
    int per_p, per_s;         // units a worker: of the prefix, of the requests
    int n_p;                  // CTAs on the prefix; the rest are on the requests
    int blocks;               // prefix: row blocks
    int chunk, chunks;        // prefix: tiles an item (the last chunk's may have fewer), items a row block
    int bad;                  // a request has more rows than max_seqlen
    int mode_s;               // the requests' mode (see few_items)
    int pad[8];
};

struct PfArgs {
    const int *table, *kv_lens, *cu, *prefix_table;
    const __nv_bfloat16* q;
    long long q_stride;
    DevStatus* status;
    PfHeader* hdr;
    PfRow* rows;              // [T]
    float *o_p, *o_s;         // segments' rows [segment][rows][D]: prefix, requests
    float2 *ml_p, *ml_s;      // their (m, l)
    void* o;
    float* lse;
    int T, B, Hq, Hkv, G, W, P, ps_log2, prefix_len, max_seqlen;
    int tq, tb;               // tokens a row tile, a row block
    int rows_p, rows_s;       // rows a segment keeps
    int tiles_p, blocks_p;    // prefix: tiles an item, row blocks
    int mode_p, mode_s;       // kFew, kOne or kTwo (see above)
    int width_p, width_s;     // workers a CTA
    int halves_p, halves_s;   // kFew: 16-row halves of a block, a warp each
    int ulog_p, ulog_s;       // log2 of the keys a unit
    // An item of a request counts its units and this many more: with 128-row
    // tiles its Q, its epilogue and the pipeline's refill cost about two tiles
    // (5000 cycles with one row tile at d = 256, 7000 with two), with few rows
    // less than one unit of 64 keys.
    int over_s;
    // A request with at least merge_n rows (four row blocks: the last one's empty
    // rows are a fifth of its work at most) takes the prefix's tiles before its own
    // ones; an item with all of its row block's tiles writes the output itself
    // (direct: this call's items can).
    int merge_n, direct, listed;   // listed: room for the prefix's row blocks in shared memory
    int qstep_p, qstep_s;     // rows between Q slots: a block's rows, in whole swizzle atoms
    float scale_log2;
};

enum : int { kPfQEmpty = 61, kPfRingEmpty, kPfQFull, kPfRingFull, kPfP, kPfS, kPfO, kPfPV, kPfDesc, kPfDescEmpty };

// ------------------------------------------------------------------ the list

// The bounded wait of every pipeline here (2 s), by a whole warp.  It looks at
// this CTA's flag alone, which takes the site that gave up, and the CTA reports it
// as it ends: a failure that an earlier call left in the device's status word does
// not stop this one.
struct PfWait {
    volatile int* abort_flag;   // shared
};
__device__ __forceinline__ bool pf_try_wait_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity), "r"(1000000u) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, const PfWait& w, int site) {
    const uint32_t a = smem_u32(bar);
    bool ok = mbar_try_wait(a, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (!(ok = pf_try_wait_long(a, parity))) {
            if (*w.abort_flag) break;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *w.abort_flag = site;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

struct Item {
    const int* tab;
    int hk, tok0, ntok, j0, j1, nkeys, lim0;
    int seg;
    int pt, whole; // tiles of the prefix before its own; 1: all its tiles are here and nothing else joins them
};

// What the roles need to know of one tile.
struct Desc {
    int page[8];            // its parts' pages, -1: none
    int live;               // one bit a part that has a page
    int flags;              // kMore (not the list's end), kFirst, kLast of its item's tiles here
    int j, nkeys, lim0, hk, tok0, ntok, seg;
};
constexpr int kMore = 1, kFirst = 2, kLast = 4, kRagged = 8, kWhole = 16;   // kRagged: some of its V rows hold no key of the list; kWhole: see Item
constexpr int kDesc = 8;    // tiles the walkers run ahead by
constexpr int kQMax = 8;    // Q slots

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Item k of a request's row blocks: from both ends by turns, so that under the
// causal mask two neighbours cost what any other two do.
__device__ __forceinline__ int block_of(int k, int n) { return (k & 1) ? n - 1 - (k >> 1) : k >> 1; }
__device__ __forceinline__ int index_of(int rb, int n) { return rb < (n + 1) / 2 ? 2 * rb : 2 * (n - 1 - rb) + 1; }

// Tiles of the prefix that the items of a request with n rows begin with.
// M: the build of the kernel for calls that can have such requests; the other has
// no trace of them (single tokens begin 2 to 4 us of a step's 50 earlier with it).
template <bool M>
__device__ __forceinline__ int prefix_tiles(const PfArgs& a, int n) { return M && n >= a.merge_n ? a.tiles_p : 0; }
// Units an item of a request with n rows and s keys has (0: no rows or no
// keys): the tiles that its row blocks see under the causal mask, on average,
// and what an item costs besides.  Row blocks are taken from both ends by turns
// (block_of), so two neighbours make up two averages.
template <bool M>
__device__ __forceinline__ int units_of(const PfArgs& a, int n, int s) {
    if (n <= 0) return 0;
    const int seen = s > 0 ? min(s, max(1, s - n + (n + min(n, a.tb)) / 2)) : 0;
    const int tiles = prefix_tiles<M>(a, n) + ((seen + (1 << a.ulog_s) - 1) >> a.ulog_s);
    return tiles > 0 ? tiles + a.over_s : 0;
}
template <int D, bool M>
__device__ __forceinline__ int item_units(const PfArgs& a, const PfTables& t, int b, int& n, int& nb) {
    n = t.cu[b + 1] - t.cu[b];
    nb = cdiv(n, a.tb);
    return units_of<M>(a, n, t.len[b]);
}
// Where unit u of an item's `units` falls among its `tiles`.
__device__ __forceinline__ int tile_of(int u, int units, int tiles) { return (int)((long long)u * tiles / units); }

// Workers a CTA on the requests.
template <int D>
__device__ __forceinline__ int width_s(const PfArgs& a, const PfHeader& h) { return D == 256 && h.mode_s == kOne ? 1 : a.width_s; }

// A worker's walk over its range of units.  Everything fits 32 bits: the host
// refuses longer lists.
template <int D, bool M>
struct Walk {
    int u, end;
    int b, hk, k, worker, chunk, chunks, blocks;
    bool pre;

    // Worker `x` of this CTA.
    __device__ __forceinline__ void start(const PfArgs& a, const PfTables& t, const PfHeader& h, int x) {
        const int c = blockIdx.x;
        b = hk = k = 0;
        chunk = h.chunk;
        chunks = h.chunks;
        blocks = h.blocks;
        pre = c < h.n_p;
        const int width = pre ? a.width_p : width_s<D>(a, h);
        worker = (pre ? c : c - h.n_p) * width + x;
        const int per = pre ? h.per_p : h.per_s, all = pre ? a.Hkv * h.blocks * a.tiles_p : t.pref[a.B];
        // worker * per passes the list's end by at most a CTA count times per.
        u = worker >= (all + per - 1) / per ? all : worker * per;
        end = min(all - u, per) + u;
        if (h.bad || x >= width || u >= end) {
            u = end = 0;
            return;
        }
        if (pre) return;
        int lo = 0, hi = a.B - 1;   // the request whose units hold u
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (t.pref[mid + 1] > u) hi = mid; else lo = mid + 1;
        }
        b = lo;
        int n, nb;
        const int per_item = item_units<D, M>(a, t, b, n, nb), i = (u - t.pref[b]) / per_item;
        hk = nb == 1 ? i : i / nb;
        k = i - hk * nb;
    }

    __device__ __forceinline__ bool next(const PfArgs& a, const PfTables& t, Item& it) {
        while (u < end) {
            if (pre) {
                // Key/value head, chunk of tiles, row block, tile: with chunks of
                // a worker's share all workers are at the same offset within
                // their chunks at a time, so the row blocks of a chunk read its
                // pages together and L2 serves all but the first.
                const int per_head = blocks * a.tiles_p;
                it.hk = u / per_head;
                const int r = u - it.hk * per_head, ch = r / (chunk * blocks);
                const int r2 = r - ch * chunk * blocks, len = min(chunk, a.tiles_p - ch * chunk);
                const int rb = r2 / len, off = r2 - rb * len, i = (it.hk * chunks + ch) * blocks + rb;
                it.j0 = ch * chunk + off;
                it.j1 = it.j0 + min(len - off, end - u);
                u += it.j1 - it.j0;
                it.tok0 = (M && t.block ? t.block[rb] : rb) * a.tb;
                it.ntok = min(a.tb, a.T - it.tok0);
                it.nkeys = a.prefix_len;
                it.lim0 = INT_MAX / 2;
                it.tab = a.prefix_table;
                it.seg = i + worker;
                it.pt = it.whole = 0;
                return true;
            }
            int n, nb;
            const int per_item = item_units<D, M>(a, t, b, n, nb), s = t.len[b];
            const int i = hk * nb + k;
            const int first = u - (t.pref[b] + i * per_item), last = min(per_item, first + end - u);
            u += last - first;
            const int i0 = block_of(k, nb) * a.tb;
            it.hk = hk;
            it.tok0 = t.cu[b] + i0;
            it.ntok = min(a.tb, n - i0);
            it.nkeys = s;
            it.lim0 = s - n + i0 + 1;
            it.tab = a.table + (long long)b * a.W;
            it.seg = t.items[b] + i + worker;
            const int seen = it.lim0 + it.ntok - 1;        // keys the block's last row sees
            it.pt = prefix_tiles<M>(a, n);
            const int tiles = it.pt + (seen > 0 ? (seen + (1 << a.ulog_s) - 1) >> a.ulog_s : 0);
            it.j0 = tile_of(first, per_item, tiles);
            it.j1 = tile_of(last, per_item, tiles);
            it.whole = M && (it.pt > 0 || a.tiles_p == 0) && it.j0 == 0 && it.j1 == tiles;
            if (last == per_item) {
                if (++k == nb) {
                    k = 0;
                    if (++hk == a.Hkv) {
                        hk = 0;
                        do ++b; while (b < a.B && t.pref[b + 1] == t.pref[b]);
                    }
                }
            }
            if (it.j0 < it.j1) return true;
        }
        return false;
    }
};

// Barriers, by their arrival counts.
struct PfShared {
    Desc desc[2][kDesc];
    // One arrival a phase.
    uint64_t d_full[2][kDesc], d_empty[2][kDesc], q_full[kQMax], q_empty[kQMax], full[8], empty[8], s_full[2], pv_done[2], o_done[2], drain[2];
    // Four: the warps of a softmax warpgroup.
    uint64_t p_ready[2], q_ready;
    // One again: few rows, each warp's slots.
    uint64_t few_full[8][12];
    Item few_item[8][2];
    int few_walk[8][12];
    int4 scan[12];
    uint32_t tmem_base;
    int abort_flag, bad;
};

// The tables of the list, by every thread of the block: the offsets by the
// library's one rule, units and items before each request, and how many CTAs
// work on the prefix.  Three block barriers when the offsets are well formed
// and B <= 384: a single-token call's latency begins here.
template <int D, bool M>
__device__ __forceinline__ PfHeader build_tables(const PfArgs& a, const PfTables& t, PfShared& sh, int tid) {
    constexpr int kThreads = Pf<D>::kThreads, kWarps = kThreads / 32;
    const int lane = tid & 31, warp = tid >> 5;
    const long long cap = (long long)a.W << a.ps_log2;
    bool fine = true;
    for (int i = tid; i <= a.B; i += kThreads) {
        const int c = a.cu ? a.cu[i] : i, before = a.cu && i > 0 ? a.cu[i - 1] : 0;
        fine = fine && c >= before && c >= 0 && c <= a.T;
        t.cu[i] = c;
        if (i < a.B) {
            const int s = a.kv_lens[i];
            t.len[i] = s < 0 ? 0 : (s > cap ? (int)cap : s);
        }
    }
    if (tid == 0) sh.bad = 0;
    if (!__syncthreads_and(fine)) {
        // Clamped to [0, T] and raised to the one before: a running maximum.
        if (warp == 0) {
            int run = 0;
            for (int base = 0; base <= a.B; base += 32) {
                int c = base + lane <= a.B ? t.cu[base + lane] : 0;
                c = c < 0 ? 0 : (c > a.T ? a.T : c);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, c, o);
                    if (lane >= o) c = max(c, x);
                }
                c = max(c, run);
                if (base + lane <= a.B) t.cu[base + lane] = c;
                run = __shfl_sync(0xffffffffu, c, 31);
            }
        }
        __syncthreads();
    }
    int units = 0, items = 0, blocks = 0;      // of the requests before these
    for (int base = 0; base < a.B; base += kThreads) {
        const int i = base + tid;
        int u = 0, it = 0, blk = 0, first_blk = 0;
        if (i < a.B) {
            int n, nb;
            const int per = item_units<D, M>(a, t, i, n, nb);
            if (n > a.max_seqlen) sh.bad = 1;
            it = nb * a.Hkv;
            u = per * it;
            if (M && t.block && n > 0 && !prefix_tiles<M>(a, n)) {
                // Row blocks of this request's rows that no request before it,
                // whose rows share the prefix too, has listed.
                first_blk = t.cu[i] / a.tb;
                blk = (t.cu[i + 1] - 1) / a.tb - first_blk + 1;
                for (int j = i - 1; j >= 0 && t.cu[j + 1] > first_blk * a.tb; --j) {
                    const int m = t.cu[j + 1] - t.cu[j];
                    if (m > 0 && !prefix_tiles<M>(a, m)) {
                        ++first_blk;
                        --blk;
                        break;
                    }
                }
            }
        }
        const int u_own = u, it_own = it, blk_own = blk;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, u, o), y = __shfl_up_sync(0xffffffffu, it, o), z = M ? __shfl_up_sync(0xffffffffu, blk, o) : 0;
            if (lane >= o) {
                u += x;
                it += y;
                if (M) blk += z;
            }
        }
        if (base) __syncthreads();
        if (lane == 31) sh.scan[warp] = make_int4(u, it, blk, 0);
        __syncthreads();
        // The warps' sums, a lane each.
        int4 all = lane < kWarps ? sh.scan[lane] : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, all.x, o), y = __shfl_up_sync(0xffffffffu, all.y, o), z = M ? __shfl_up_sync(0xffffffffu, all.z, o) : 0;
            if (lane >= o) {
                all.x += x;
                all.y += y;
                if (M) all.z += z;
            }
        }
        auto sum_of = [&](int x, int w) { return __shfl_sync(0xffffffffu, x, w); };
        const int u_all = sum_of(all.x, kWarps - 1), it_all = sum_of(all.y, kWarps - 1), blk_all = M ? sum_of(all.z, kWarps - 1) : 0;
        const int u_before = sum_of(all.x, max(warp - 1, 0)), it_before = sum_of(all.y, max(warp - 1, 0)), blk_before = M ? sum_of(all.z, max(warp - 1, 0)) : 0;
        u += units + (warp ? u_before : 0);
        it += items + (warp ? it_before : 0);
        if (M) blk += blocks + (warp ? blk_before : 0);
        if (i < a.B) {
            t.pref[i] = u - u_own;
            t.items[i] = it - it_own;
            if (M)
                for (int k = 0; k < blk_own; ++k) t.block[blk - blk_own + k] = first_blk + k;
        }
        units += u_all;
        items += it_all;
        blocks += blk_all;
    }
    if (tid == 0) {
        t.pref[a.B] = units;
        t.items[a.B] = items;
    }
    __syncthreads();
    PfHeader h;
    h.mode_s = a.mode_s == kFew && !Pf<D>::few_items(units, items) ? kOne : a.mode_s;
    h.blocks = M && t.block ? blocks : a.blocks_p;
    const int grid = gridDim.x, units_p = a.Hkv * h.blocks * a.tiles_p;
    const float keys_p = (float)units_p * (1 << a.ulog_p), keys_s = (float)units * (1 << a.ulog_s);
    const float cp = (float)units_p * Pf<D>::cost_p(a.mode_p, a.halves_p, h.blocks > 1, keys_s / fmaxf(keys_p + keys_s, 1.f));
    const float cs = (float)units * Pf<D>::cost_s(h.mode_s, a.halves_s);
    int np = units_p == 0 ? 0 : (units == 0 ? grid : (int)(grid * (cp / (cp + cs)) + 0.5f));
    if (units_p > 0 && units > 0) np = max(1, min(grid - 1, np));
    int wp = np * a.width_p;
    h.per_p = wp ? (units_p + wp - 1) / wp : 1;
    // Chunks are a worker's share of tiles; a small rest would be a chunk of its
    // own in every row block (62 tiles a worker of 256: 135 us for 100 rows of 32
    // heads at d = 256, 64: 104), so it is spread over the others.
    if (h.blocks > 1 && units > 0 && a.tiles_p > h.per_p && a.tiles_p % h.per_p < h.per_p / 4) {
        const int k = a.tiles_p / h.per_p;
        h.per_p = (a.tiles_p + k - 1) / k;
        np = max(1, min(np, cdiv(units_p, h.per_p * a.width_p)));
    }
    const int ws = max(1, grid - np) * width_s<D>(a, h);
    h.n_p = np;
    h.per_s = units ? (units + ws - 1) / ws : 1;
    h.chunk = h.blocks > 1 ? max(1, min(h.per_p, a.tiles_p)) : max(1, a.tiles_p);
    h.chunks = (a.tiles_p + h.chunk - 1) / h.chunk;
    h.bad = sh.bad;
    if (blockIdx.x == 0 && tid == 0) {
        *a.hdr = h;
        if (h.bad && atomicCAS(&a.status->code, 0, -1) == 0) { a.status->where = 101; a.status->block = 0; }
    }
    return h;
}

// ------------------------------------------------------------------ products

// Q from shared memory, at d = 256 from tensor memory: a 128 x 64 x 16 product with
// both operands in shared memory is bound by its bandwidth (48 cycles, not 32).
template <int D>
__device__ __forceinline__ void pf_issue_qk(uint32_t d_tmem, uint32_t q, uint32_t k_smem) {
    using G = Pf<D>;
    constexpr uint32_t idesc = idesc_bf16_f32(128, G::kN, 0, 0);
    const uint64_t qd = sdesc_sw128(q, 16, 1024), kd = sdesc_sw128(k_smem, 16, 1024);
    static_for<D / 16>([&](auto kc) {
        constexpr uint32_t k = kc;
        constexpr uint32_t ao = ((k >> 2) * G::kQBox + (k & 3) * 32) >> 4, bo = ((k >> 2) * G::kKVBox + (k & 3) * 32) >> 4;
        if constexpr (D == 256) umma_ts_k<k * 8, bo>(d_tmem, q, kd, idesc, k > 0);
        else umma_ss_k<ao, bo>(d_tmem, qd, kd, idesc, k > 0);
    });
}

template <int D>
__device__ __forceinline__ void pf_issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_smem, uint32_t acc) {
    using G = Pf<D>;
    constexpr uint32_t idesc = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t vd = sdesc_sw128(v_smem, G::kKVBox, 1024);
    static_for<G::kN / 16>([&](auto kc) {
        constexpr uint32_t k = kc;
        umma_ts_k<k * 8, ((k * 2048) >> 4)>(d_tmem, p_tmem, vd, idesc, (acc | k) != 0);
    });
}

// ------------------------------------------------------------------ few rows
//
// Blocks of at most 32 rows (single tokens, small drafts): the copies set the
// pace, and what a 128-row product would cost is synchronisation (S, P and O
// pass between three roles for every tile) and a softmax that one warp in four
// would run.  Here each of eight warps is a worker of its own, or each pair of
// warps when there are more than 16 rows (each takes 16): it walks its range of
// the list, copies 16 keys of K or V at a time into a ring of its own
// (TMA; a slot is free as soon as this warp has read it, so nothing waits for
// another warp), and keeps scores, weights and the accumulator in registers
// (mma.sync m16n8k16).  An item's end costs a store of the rows and no barrier.
// A step is 8 KB of K and of V (64 keys at d = 64, 16 at d = 256, where Q and O
// take the registers).  For 64 keys a CTA's eight warps take 780 to 880 cycles at d
// = 128 while a third of the CTAs copy (37 to 42 B a cycle; an equal share of HBM
// for all is 23), 520 at d = 64 (with 32 keys a step 600: 32 requests of 32 heads 58
// us, with 64 49).  64 single tokens with 4000 to 16000 keys of their own and no
// prefix: 6.8 TB/s.  Eight warps that share 128-key tiles and join in shared memory
// took 442 us where these take 349.

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool M>
__device__ __forceinline__ void few_rows(const CUtensorMap* tk, const CUtensorMap* tv, const PfArgs& a, const PfTables& t,
                                         const PfHeader& hdr, PfShared& sh, uint32_t smem, const PfWait& wc, bool pre, int warp, int lane) {
    using G = Pf<D>;
    constexpr int kKT = G::kFewParts, kKeys = 16 * kKT;              // 16-key parts and keys a step
    constexpr uint32_t kPart = D * 32u, kSlot = kPart * kKT;         // K or V of a part (D / 64 boxes of 16 x 128 B), of a step
    constexpr uint32_t kRing = G::kFewRing;
    constexpr int kKSteps = D / 16, kNT = D / 8;
    const int halves = pre ? a.halves_p : a.halves_s, half = warp % halves, ulog = pre ? a.ulog_p : a.ulog_s;
    const int g = lane >> 2, t2 = (lane & 3) * 2;
    // ldmatrix: this lane's row of the four 8 x 8 matrices and which 16-byte
    // chunk of each 32-byte step it is; chunks are swizzled by row % 8 within a
    // 128-byte row.
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t ring = smem + warp * (kRing * kSlot);
    const uint32_t k_row = ((mi >> 1) * 8 + mr) * 128u, v_row = ((mi & 1) * 8 + mr) * 128u;
    const float scale = a.scale_log2;
    uint64_t* full = sh.few_full[warp];

    // The walk and the two items that the warp knows (the one it works on and
    // the next, by turns) stay in shared memory: registers go to Q and O.
    Walk<D, M>* walk = reinterpret_cast<Walk<D, M>*>(sh.few_walk[warp]);
    Item* items = sh.few_item[warp];
    {
        Walk<D, M> w;
        w.start(a, t, hdr, warp / halves);
        if (lane == 0) *walk = w;
        __syncwarp();
    }
    // 16-key parts of an item: up to its last row's last key.
    auto parts_of = [&](const Item& it) {
        return (min(min(it.j1 << ulog, it.nkeys), it.lim0 + it.ntok - 1) - (it.j0 << ulog) + 15) >> 4;
    };
    // This half's next item (one without rows for it is skipped) into items[to].
    auto next_item = [&](int to) -> bool {
        Walk<D, M> w = *walk;
        Item it;
        bool more;
        do more = w.next(a, t, it); while (more && half * 16 >= it.ntok * a.G);
        __syncwarp();
        if (lane == 0) {
            *walk = w;
            if (more) items[to] = it;
        }
        __syncwarp();
        return more;
    };
    // Pages of 32 parts of an item, one a lane.
    auto pages = [&](const Item& it, int s0) -> int {
        if (s0 + lane >= parts_of(it)) return -1;
        const int p = it.tab[((it.j0 << ulog) + (s0 + lane) * 16) >> a.ps_log2];
        return p >= 0 && p < a.P ? p : -1;
    };
    // The copies run ahead of the work, at most into the next item.
    int cur = 0;                                                     // items[cur], items[cur ^ 1] is the next
    bool has_next = false, in_next = false;                          // it is known; the copies are in it
    int copy_part = 0, copy_parts = 0, copy_pg = -1, copy_hk = 0, copy_key = 0;   // next part in their item, its parts, this lane's page, head, key
    int win = -1, ahead = -1, first = -1;                            // pages: of their 32 parts, of the next 32, of the next item's first 32
    uint32_t issued = 0, filled = 0, live_bits = 0;                  // slots filled, the next one; one bit a part (mod 32): its page exists
    bool ok = true;
    auto enter = [&](const Item& it) {                               // the copies begin an item
        copy_part = 0;
        copy_parts = parts_of(it);
        copy_hk = it.hk;
        copy_key = it.j0 << ulog;
        win = first;
        ahead = pages(it, 32);
    };
    // Fills the next slot (K, then V of a step) if there is a step left to copy.
    // Lane i copies part i.
    auto copy = [&]() {
        if (!(issued & 1)) {                                         // a new step
            if (copy_part >= copy_parts) {
                if (in_next || !has_next) return;
                in_next = true;
                enter(items[cur ^ 1]);
            } else if (copy_part > 0 && (copy_part & 31) == 0) {
                win = ahead;
                ahead = pages(items[in_next ? cur ^ 1 : cur], copy_part + 32);
            }
            copy_pg = __shfl_sync(0xffffffffu, win, (copy_part + (lane & (kKT - 1))) & 31);   // -1 past the item's end
            const uint32_t live = __ballot_sync(0xffffffffu, copy_pg >= 0) & ((1u << kKT) - 1u), at = (issued >> 1) * kKT & 31;
            live_bits = (live_bits & ~(((1u << kKT) - 1u) << at)) | live << at;
        }
        const uint32_t live = live_bits >> ((issued >> 1) * kKT & 31) & ((1u << kKT) - 1u);
        uint64_t* bar = &full[filled];
        __syncwarp();                                                // every lane has read what the slot held
        if (lane == 0) {
            if (live) mbar_arrive_expect_tx(bar, kPart * __popc(live));
            else mbar_arrive(bar);
        }
        __syncwarp();
        if (lane < kKT && copy_pg >= 0)
            tma_load_3d(ring + filled * kSlot + lane * kPart, issued & 1 ? tv : tk, bar, 0,
                        ((copy_pg * a.Hkv + copy_hk) << a.ps_log2) + ((copy_key + (copy_part + lane) * 16) & ((1 << a.ps_log2) - 1)), 0);
        if (issued & 1) copy_part += kKT;
        ++issued;
        filled = filled + 1 == kRing ? 0 : filled + 1;
    };

    uint32_t n = 0, slot = 0, phase = 0;                             // slots read, the next one, its barrier's parity
    auto wait = [&]() { return pf_wait(&full[slot], phase, wc, kPfRingFull); };
    auto next_slot = [&]() {
        ++n;
        if (++slot == kRing) {
            slot = 0;
            phase ^= 1;
        }
    };
    if (next_item(0)) {
        first = pages(items[0], 0);
        enter(items[0]);
        if ((has_next = next_item(1))) first = pages(items[1], 0);
        for (uint32_t i = 0; i < kRing; ++i) copy();
        while (ok) {
            const Item& it = items[cur];
            const int parts = parts_of(it), nkeys = it.nkeys, key0 = it.j0 << ulog;
            // Q as A fragments, straight from memory; rows without a query are 0.
            uint32_t qf[kKSteps][4];
            float o[kNT][4], m[2], l[2];
            int lim[2];
            const int rows = it.ntok * a.G;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = half * 16 + h * 8 + g, tok = r / a.G;
                const bool real = r < rows;
                lim[h] = !real ? 0 : pre ? it.nkeys : min(it.nkeys, it.lim0 + tok);
                m[h] = -INFINITY;
                l[h] = 0.f;
                const __nv_bfloat16* src = a.q + (long long)(it.tok0 + tok) * a.q_stride + (it.hk * a.G + r - tok * a.G) * D + t2;
#pragma unroll
                for (int ks = 0; ks < kKSteps; ++ks) {
                    qf[ks][h] = real ? *reinterpret_cast<const uint32_t*>(src + ks * 16) : 0u;
                    qf[ks][2 + h] = real ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8) : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < kNT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            const int lim_min = pre ? it.nkeys : min(it.nkeys, it.lim0 + half * 16 / a.G);
            for (int st = 0; st < parts; st += kKT) {
                const int k0 = key0 + st * 16;
                const uint32_t live = live_bits >> ((n >> 1) * kKT & 31) & ((1u << kKT) - 1u);
                uint32_t p[kKT][4];
                if (!(ok = wait())) break;
                if (live) {
                    float s[2 * kKT][4] = {};
                    const uint32_t base = ring + slot * kSlot + k_row;
                    // Four loads, then their eight products: a load's latency
                    // (33 cycles) is paid once a batch.
                    constexpr int kBatch = 4 / kKT;
#pragma unroll
                    for (int k4 = 0; k4 < kKSteps; k4 += kBatch) {
                        uint32_t b[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ks = k4 + i / kKT, kt = i % kKT;
                            ldsm4(b[i], base + kt * kPart + (ks >> 2) * 2048u + (((((ks & 3) << 1) + (mi & 1)) ^ mr) << 4));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ks = k4 + i / kKT, kt = i % kKT;
                            mma16816(s[2 * kt], qf[ks], b[i][0], b[i][1]);
                            mma16816(s[2 * kt + 1], qf[ks], b[i][2], b[i][3]);
                        }
                    }
                    if (k0 + kKeys > lim_min || live != (1u << kKT) - 1u) {
#pragma unroll
                        for (int i = 0; i < 2 * kKT; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!((live >> (i >> 1)) & 1u) || k0 + i * 8 + t2 + (e & 1) >= lim[e >> 1]) s[i][e] = -INFINITY;
                    }
                    float mn[2];
                    bool jump = false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = fmaxf(s[0][2 * h], s[0][2 * h + 1]);
#pragma unroll
                        for (int i = 1; i < 2 * kKT; ++i) x = fmax3(x, s[i][2 * h], s[i][2 * h + 1]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        mn[h] = fmaxf(m[h], x * scale);
                        jump |= (m[h] == -INFINITY) ? (mn[h] != -INFINITY) : (mn[h] - m[h] > kTau);
                    }
                    if (__any_sync(0xffffffffu, jump)) {
                        float fac[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            fac[h] = m[h] == -INFINITY ? 0.f : ex2_mufu(m[h] - mn[h]);
                            l[h] *= fac[h];
                            m[h] = mn[h];
                        }
#pragma unroll
                        for (int i = 0; i < kNT; ++i) {
                            o[i][0] *= fac[0];
                            o[i][1] *= fac[0];
                            o[i][2] *= fac[1];
                            o[i][3] *= fac[1];
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float use = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
                        for (int i = 0; i < 2 * kKT; ++i) {
                            const float p0 = ex2_mufu(fmaf(s[i][2 * h], scale, -use)), p1 = ex2_mufu(fmaf(s[i][2 * h + 1], scale, -use));
                            l[h] += p0 + p1;
                            p[i >> 1][2 * (i & 1) + h] = pack_bf16x2(p0, p1);   // 16-bit weights feed the product; l keeps 32 bits
                        }
                    }
                }
                next_slot();
                copy();
                if (!(ok = wait())) break;
                if (live) {
                    const uint32_t base = ring + slot * kSlot + v_row;
                    // Keys behind the list's end and of absent pages count as 0,
                    // whatever their rows hold.
                    auto pair = [&](int key) { return (key < nkeys ? 0xffffu : 0u) | (key + 1 < nkeys ? 0xffff0000u : 0u); };
                    const bool whole = k0 + kKeys <= nkeys && live == (1u << kKT) - 1u;
#pragma unroll
                    for (int kt = 0; kt < kKT; ++kt) {
                        const uint32_t here = (live >> kt) & 1u ? ~0u : 0u;
                        const uint32_t w0 = whole ? ~0u : here & pair(k0 + kt * 16 + t2), w1 = whole ? ~0u : here & pair(k0 + kt * 16 + 8 + t2);
#pragma unroll
                        for (int i4 = 0; i4 < kNT; i4 += 8) {
                            uint32_t b[4][4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int i = i4 + 2 * e;
                                ldsm4t(b[e], base + kt * kPart + (i >> 3) * 2048u + ((((i & 7) + (mi >> 1)) ^ mr) << 4));
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int i = i4 + 2 * e;
                                mma16816(o[i], p[kt], b[e][0] & w0, b[e][1] & w1);
                                mma16816(o[i + 1], p[kt], b[e][2] & w0, b[e][3] & w1);
                            }
                        }
                    }
                }
                next_slot();
                copy();
            }
            if (!ok) break;
            // The rows' (m, l, O) into the segment's place.
            const long long at = (long long)it.seg * (pre ? a.rows_p : a.rows_s);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int r = half * 16 + h * 8 + g;
                if (r < rows) {
                    float* out = (pre ? a.o_p : a.o_s) + (at + r) * D + t2;
#pragma unroll
                    for (int i = 0; i < kNT; ++i) *reinterpret_cast<float2*>(out + i * 8) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
                    if (t2 == 0) (pre ? a.ml_p : a.ml_s)[at + r] = make_float2(m[h], l[h]);
                }
            }
            if (!has_next) break;
            // The next item becomes this one.
            cur ^= 1;
            if (in_next) in_next = false;
            else enter(items[cur]);
            if ((has_next = next_item(cur ^ 1))) first = pages(items[cur ^ 1], 0);
            while (issued - n < kRing) {
                const uint32_t before = issued;
                copy();
                if (issued == before) break;
            }
        }
    }
    // Every copy lands before teardown (after a wait that gave up, too).
    const uint64_t t0 = globaltimer_ns();
    for (; n < issued; next_slot())
        while (!mbar_try_wait(smem_u32(&full[slot]), phase) && globaltimer_ns() - t0 < kWaitLimitNs) {}
    __syncwarp();
}

// -------------------------------------------------------------------- kernel

template <int D, bool M>
__global__ void __launch_bounds__(Pf<D>::kThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap tq_p, const __grid_constant__ CUtensorMap tq_s,
              const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
              const __grid_constant__ CUtensorMap tk_few, const __grid_constant__ CUtensorMap tv_few, const PfArgs a) {
    using G = Pf<D>;
    constexpr int kN = G::kN, kStreams = G::kStreams, kRing = G::kRing, kBoxes = G::kBoxes;
    constexpr int kSoftWarps = 8;
    extern __shared__ uint8_t dsmem[];
    __shared__ PfShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
    uint8_t* gbase = dsmem + (base - smem_u32(dsmem));
    const uint32_t sQ = base, sRing = base + G::kStreams * G::kQTile;
    PfTables t;
    t.pref = reinterpret_cast<int*>(gbase + G::kTiles);
    t.items = reinterpret_cast<int*>(t.pref + a.B + 1);
    t.cu = t.items + a.B + 1;
    t.len = t.cu + a.B + 1;
    t.block = M && a.merge_n < INT_MAX ? t.len + a.B : nullptr;

    {   // One barrier a thread, in the order of PfShared.
        constexpr int n1 = (offsetof(PfShared, p_ready) - offsetof(PfShared, d_full)) / 8;
        constexpr int n4 = (offsetof(PfShared, few_full) - offsetof(PfShared, p_ready)) / 8;
        constexpr int nf = (offsetof(PfShared, few_item) - offsetof(PfShared, few_full)) / 8;
        static_assert(n1 + n4 + nf <= G::kThreads, "one barrier a thread");
        static_assert(sizeof(Walk<D, M>) <= sizeof(PfShared::few_walk[0]) && G::kFewRing <= 12, "few rows");
        if (tid < n1 + n4 + nf) {
            mbar_init(&sh.d_full[0][0] + tid, tid >= n1 && tid < n1 + n4 ? 4 : 1);
            fence_mbar_init();
        }
        if (tid == 0) sh.abort_flag = 0;
    }
    if (warp == kSoftWarps + 3) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    grid_launch_next();
    grid_wait();
    const PfHeader hdr = build_tables<D, M>(a, t, sh, tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const PfWait wc{&sh.abort_flag};
    const uint32_t tmem = sh.tmem_base;
    // Parts of a tile: whole pages, or one part where a page is larger.
    const int part_log2 = min(a.ps_log2, kN == 64 ? 6 : 7), parts = kN >> part_log2;
    const bool pre = (int)blockIdx.x < hdr.n_p;
    const int mode = pre ? a.mode_p : hdr.mode_s;
    const bool two = kStreams == 2 && mode == kTwo, few = mode == kFew;
    const int workers = two ? 1 : kStreams;
    // Q slots: two row tiles, one slot of both; else as many in a worker's row
    // tile as its rows (in whole swizzle atoms) leave room for.  The products
    // read 128 rows from a slot on; the rows past its own give scores that
    // nobody looks at.
    const int qstep = pre ? a.qstep_p : a.qstep_s;
    const uint32_t qn = two ? 1 : min(kQMax / kStreams, 128 / qstep);
    auto q_slot = [&](int x, uint32_t item) { return two ? 0u : x * qn + item % qn; };
    auto q_addr = [&](int x, uint32_t item) { return sQ + x * G::kQTile + (two ? 0u : (item % qn) * qstep * 128u); };
    auto desc_wait = [&](int x, uint32_t n) { return pf_wait(&sh.d_full[x][n % kDesc], (n / kDesc) & 1, wc, kPfDesc); };

    // What the joining kernel needs to know of each row.
    auto owners = [&]() {
        if (warp != kSoftWarps + 3) return;
        for (int i = blockIdx.x * 32 + lane; i < a.T; i += gridDim.x * 32) {
            PfRow row = {};
            if (i >= t.cu[0] && i < t.cu[a.B]) {
                int lo = 0;
                for (int hi = a.B; hi - lo > 1;) {   // the last request that begins at or before i
                    const int mid = (lo + hi) >> 1;
                    if (t.cu[mid] <= i) lo = mid; else hi = mid;
                }
                row.c0 = t.cu[lo];
                row.n = t.cu[lo + 1] - row.c0;
                row.s = t.len[lo];
                row.pref = t.pref[lo];
                row.items = t.items[lo];
                row.block = a.tiles_p == 0 || prefix_tiles<M>(a, row.n) ? -1 : i / a.tb;
                if (M && t.block && row.block >= 0) {
                    int at = 0;
                    for (int hi = hdr.blocks; hi - at > 1;) {
                        const int mid = (at + hi) >> 1;
                        if (t.block[mid] <= row.block) at = mid; else hi = mid;
                    }
                    row.block = at;
                }
            }
            a.rows[i] = row;
        }
        __syncwarp();
    };
    // Registers: 384 x 168 at launch, moved to the warpgroups that compute
    // (2 x 232 + 40 or 2 x 208 + 88 = 3 x 168).
    if (few) {
        if (warp >= kSoftWarps) {
            regs_dec<40>();
            owners();
        } else {
            regs_inc<232>();
            few_rows<D, M>(&tk_few, &tv_few, a, t, hdr, sh, base, wc, pre, warp, lane);
        }
    } else if (warp >= kSoftWarps) {
        regs_dec<88>();
        owners();
        if (warp == kSoftWarps) {
            // ------------------------------------------------------------ loader
            // The issuer's order: every worker's first K (kLook of them), then by
            // turns a worker's V of the oldest tile and K of the next one.
            // Lane i * kBoxes + c copies box c of part i (at most 16 lanes).
            uint32_t n_ring = 0, n_item[2] = {0, 0}, n_k[2] = {0, 0}, n_v[2] = {0, 0};
            bool ended[2] = {false, false};
            int pg[2][2] = {}, row[2][2] = {};               // of tiles whose V is still to come
            const int part = lane / kBoxes, col = lane % kBoxes;
            const uint32_t part_bytes = 128u << part_log2;
            bool ok = true;
            auto load = [&](const CUtensorMap* map, int p, int r) -> bool {
                const uint32_t slot = n_ring % kRing;
                if (!pf_wait(&sh.empty[slot], ((n_ring / kRing) & 1) ^ 1, wc, kPfRingEmpty)) return false;
                const uint32_t live = __ballot_sync(0xffffffffu, p >= 0);
                if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], __popc(live) * part_bytes);
                __syncwarp();
                if (p >= 0)
                    tma_load_2d(sRing + slot * G::kTile + col * G::kKVBox + part * part_bytes, map, &sh.full[slot], col * 64, r);
                ++n_ring;
                return true;
            };
            auto load_k = [&](int x) -> bool {
                if (!desc_wait(x, n_k[x])) return false;
                const Desc& d = sh.desc[x][n_k[x] % kDesc];
                const int flags = d.flags;
                if (!(flags & kMore)) {
                    ended[x] = true;
                    return true;
                }
                pg[x][1] = pg[x][0];
                row[x][1] = row[x][0];
                pg[x][0] = part < parts ? d.page[part] : -1;
                row[x][0] = ((pg[x][0] * a.Hkv + d.hk) << a.ps_log2) + ((d.j * kN + (part << part_log2)) & ((1 << a.ps_log2) - 1));
                if (!load(&tk, pg[x][0], row[x][0])) return false;
                if (kStreams == 2 && (flags & kFirst)) {
                    const uint32_t i = n_item[x], s = q_slot(x, i);
                    if (!pf_wait(&sh.q_empty[s], ((i / qn) & 1) ^ 1, wc, kPfQEmpty)) return false;
                    const int boxes = two ? 2 * kBoxes : kBoxes;
                    if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[s], boxes * 128u * a.G * min(a.tq, pre ? a.T : a.max_seqlen));
                    __syncwarp();
                    if (lane < boxes) {
                        const int tile = lane / kBoxes, c = lane % kBoxes;
                        tma_load_3d(q_addr(two ? tile : x, i) + c * G::kQBox, pre ? &tq_p : &tq_s, &sh.q_full[s], c * 64, d.hk * a.G,
                                    d.tok0 + tile * a.tq);
                    }
                    ++n_item[x];
                }
                ++n_k[x];
                return true;
            };
            for (int i = 0; i < G::kLook && ok; ++i)
#pragma unroll
                for (int x = 0; x < kStreams; ++x)
                    if (ok && x < workers && !ended[x]) ok = load_k(x);
            bool any = true;
            while (ok && any) {
                any = false;
#pragma unroll
                for (int x = 0; x < kStreams; ++x) {
                    if (!ok || n_v[x] == n_k[x]) continue;
                    any = true;
                    const bool older = n_k[x] - n_v[x] == 2;
                    if (!(ok = load(&tv, older ? pg[x][1] : pg[x][0], older ? row[x][1] : row[x][0]))) break;
                    ++n_v[x];
                    if (!ended[x]) ok = load_k(x);
                }
            }
            // Every copy lands before teardown.
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t i = n_ring > kRing ? n_ring - kRing : 0; i < n_ring; ++i)
                while (!mbar_try_wait(smem_u32(&sh.full[i % kRing]), (i / kRing) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            for (int x = 0; x < workers; ++x)
                for (uint32_t i = n_item[x] > qn ? n_item[x] - qn : 0; i < n_item[x]; ++i)
                    while (!mbar_try_wait(smem_u32(&sh.q_full[q_slot(x, i)]), (i / qn) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            __syncwarp();
        } else if (warp == kSoftWarps + 1 || (kStreams == 1 && warp == kSoftWarps + 3)) {
            // ------------------------------------------------------- UMMA issuer
            uint32_t n_ring = 0;
            bool ok = true;
            auto col_s = [&](int x) { return tmem + G::kColS + x * G::kColSStep; };
            // Waits for the next tile of the ring; its slot.
            auto take = [&](uint32_t& slot) -> bool {
                slot = n_ring % kRing;
                if (!pf_wait(&sh.full[slot], (n_ring / kRing) & 1, wc, kPfRingFull)) return false;
                ++n_ring;
                return true;
            };
            // Zeroes the V rows of a tile that hold no key of the list.
            auto clean = [&](uint32_t slot, const Desc& d) {
                const int rows = d.nkeys - d.j * kN, live = d.live;
                for (int i = 0; i < parts; ++i) {
                    const int r0 = i << part_log2, r1 = r0 + (1 << part_log2);
                    const int from = (live >> i) & 1 ? max(r0, min(r1, rows)) : r0;
                    for (int c = 0; c < kBoxes; ++c)
                        for (uint32_t o = from * 128u + lane * 16u; o < r1 * 128u; o += 512u)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                                         ::"r"(sRing + slot * G::kTile + c * G::kKVBox + o), "r"(0u) : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            };
            auto free_desc = [&](int x, uint32_t n) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.d_empty[x][n % kDesc]);
            };
            if (two) {
                if constexpr (kStreams == 2) {
                    uint32_t ks, vs, items = 0;
                    auto qk = [&](int x, int flags) {
                        pf_issue_qk<D>(col_s(x), sQ + x * G::kQTile, sRing + ks * G::kTile);
                        umma_commit_w(&sh.s_full[x]);
                        if (x == 1) {
                            umma_commit_w(&sh.empty[ks]);
                            if (flags & kLast) umma_commit_w(&sh.q_empty[0]);
                        }
                    };
                    auto new_item = [&]() -> bool { return pf_wait(&sh.q_full[0], items++ & 1, wc, kPfQFull); };
                    int flags = 0;
                    if ((ok = desc_wait(0, 0))) flags = sh.desc[0][0].flags;
                    if (ok && (flags & kMore) && (ok = take(ks)) && (ok = new_item())) {
                        qk(0, flags);
                        qk(1, flags);
                    }
                    for (uint32_t n = 0; ok && (flags & kMore); ++n) {
                        const Desc& d = sh.desc[0][n % kDesc];
                        if (!(ok = desc_wait(0, n + 1))) break;
                        const int ahead = sh.desc[0][(n + 1) % kDesc].flags;
                        if (!(ok = take(vs))) break;
                        if ((ahead & kMore) && !(ok = take(ks))) break;
                        if (flags & kRagged) clean(vs, d);
                        for (int x = 0; x < 2; ++x) {
                            if (!(ok = pf_wait(&sh.p_ready[x], n & 1, wc, kPfP))) break;
                            tc_fence_after();
                            pf_issue_pv<D>(tmem + x * G::kColO1, col_s(x), sRing + vs * G::kTile, !(flags & kFirst));
                            if (x == 1) umma_commit_w(&sh.empty[vs]);
                            if (flags & kLast) umma_commit_w(&sh.o_done[x]);
                            else qk(x, ahead);
                        }
                        if (!ok) break;
                        if ((flags & kLast) && (ahead & kMore)) {
                            if (!(ok = new_item())) break;
                            qk(0, ahead);
                            qk(1, ahead);
                        }
                        free_desc(0, n);
                        flags = ahead;
                    }
                }
            } else if constexpr (kStreams == 1) {
                // One worker, S double-buffered: S and P V have an issuer each.
                // Issuing blocks while the tensor core is busy, and one issuer's
                // waits would stand between the products of every tile (2540
                // cycles a tile with one issuer, 1280 of them products).  The
                // ring's order: K0, K1, V0, K2, V1, K3, ..., the last V behind the
                // one before.
                auto wait_tile = [&](uint32_t i) { return pf_wait(&sh.full[i % kRing], (i / kRing) & 1, wc, kPfRingFull); };
                if (warp == kSoftWarps + 3) {
                    uint32_t items = 0;
                    for (uint32_t n = 0;; ++n) {
                        if (!(ok = desc_wait(0, n))) break;
                        const int flags = sh.desc[0][n % kDesc].flags, buf = n & 1;
                        if (!(flags & kMore)) break;
                        const uint32_t i = n < 2 ? n : 2 * n - 1;
                        if ((flags & kFirst) && !(ok = pf_wait(&sh.q_ready, items++ & 1, wc, kPfQFull))) break;
                        if (!(ok = wait_tile(i))) break;
                        // S goes where P of two tiles before was read from.
                        if (n >= 2 && !(ok = pf_wait(&sh.pv_done[buf], ((n - 2) >> 1) & 1, wc, kPfPV))) break;
                        tc_fence_after();
                        pf_issue_qk<D>(col_s(buf), tmem + G::kColQ, sRing + i % kRing * G::kTile);
                        umma_commit_w(&sh.s_full[buf]);
                        umma_commit_w(&sh.empty[i % kRing]);
                        if (flags & kLast) umma_commit_w(&sh.q_empty[0]);
                    }
                } else {
                    if ((ok = desc_wait(0, 0))) {
                        int flags = sh.desc[0][0].flags;
                        for (uint32_t n = 0; flags & kMore; ++n) {
                            if (!(ok = desc_wait(0, n + 1))) break;
                            const int ahead = sh.desc[0][(n + 1) % kDesc].flags, buf = n & 1;
                            const uint32_t i = ahead & kMore ? 2 * n + 2 : 2 * n + 1;
                            if (!(ok = wait_tile(i))) break;
                            if (flags & kRagged) clean(i % kRing, sh.desc[0][n % kDesc]);
                            if (!(ok = pf_wait(&sh.p_ready[buf], (n >> 1) & 1, wc, kPfP))) break;
                            tc_fence_after();
                            pf_issue_pv<D>(tmem, col_s(buf), sRing + i % kRing * G::kTile, !(flags & kFirst));
                            umma_commit_w(&sh.pv_done[buf]);
                            umma_commit_w(&sh.empty[i % kRing]);
                            if (flags & kLast) umma_commit_w(&sh.o_done[0]);
                            free_desc(0, n);
                            flags = ahead;
                        }
                    }
                }
            } else {
                uint32_t n_s[2] = {0, 0}, n_p[2] = {0, 0}, n_item[2] = {0, 0}, ks;
                bool ended[2] = {false, false};
                // The K of worker x's next tile, if it has one (its flags, else 0).
                int flags_s = 0;
                auto take_k = [&](int x) -> bool {
                    flags_s = 0;
                    if (ended[x]) return true;
                    if (!desc_wait(x, n_s[x])) return false;
                    flags_s = sh.desc[x][n_s[x] % kDesc].flags;
                    ended[x] = !(flags_s & kMore);
                    if (ended[x]) flags_s = 0;
                    return ended[x] || take(ks);
                };
                // Its S.
                auto issue_s = [&](int x) -> bool {
                    if (flags_s & kFirst) {
                        const uint32_t i = n_item[x]++;
                        if (!pf_wait(&sh.q_full[q_slot(x, i)], (i / qn) & 1, wc, kPfQFull)) return false;
                    }
                    pf_issue_qk<D>(col_s(x), q_addr(x, n_item[x] - 1), sRing + ks * G::kTile);
                    umma_commit_w(&sh.s_full[x]);
                    umma_commit_w(&sh.empty[ks]);
                    if (flags_s & kLast) umma_commit_w(&sh.q_empty[q_slot(x, n_item[x] - 1)]);
                    ++n_s[x];
                    return true;
                };
#pragma unroll
                for (int x = 0; x < kStreams; ++x)
                    if (ok && !ended[x]) ok = take_k(x) && (!flags_s || issue_s(x));
                bool any = true;
                while (ok && any) {
                    any = false;
#pragma unroll
                    for (int x = 0; x < kStreams; ++x) {
                        if (!ok || n_p[x] == n_s[x]) continue;
                        any = true;
                        const uint32_t n = n_p[x];
                        const Desc& d = sh.desc[x][n % kDesc];
                        const int flags = d.flags;
                        uint32_t vs;
                        if (!(ok = take(vs))) break;
                        if (flags & kRagged) clean(vs, d);
                        // Both tiles are waited for before P, so that S follows P V
                        // into the tensor core without a pause.
                        if (!(ok = take_k(x))) break;
                        if (!(ok = pf_wait(&sh.p_ready[x], n & 1, wc, kPfP))) break;
                        tc_fence_after();
                        pf_issue_pv<D>(tmem + x * G::kColO1, col_s(x), sRing + vs * G::kTile, !(flags & kFirst));
                        umma_commit_w(&sh.empty[vs]);
                        if (flags & kLast) umma_commit_w(&sh.o_done[x]);
                        if (flags_s && !(ok = issue_s(x))) break;
                        free_desc(x, n);
                        ++n_p[x];
                    }
                }
            }
            // All products complete before tensor memory is freed.
            uint64_t* drain = &sh.drain[warp == kSoftWarps + 1 ? 0 : 1];
            umma_commit_w(drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            __syncwarp();
        } else if (warp - (kSoftWarps + 2) < workers) {
            // ------------------------------------------------------ list walkers
            // Pages of four tiles at a time, a lane each; the next four's loads
            // (the next item's, past an item's end) run while these are handed on.
            // The first four are handed on before any others are looked up: every
            // role waits for them.  Turns: look up 0; hand on 0; look up 1; look up 2
            // and hand on 1; look up 3 and hand on 2; ...
            const int x = warp - (kSoftWarps + 2), q = lane >> 3, part = lane & 7;
            Walk<D, M> walk;
            walk.start(a, t, hdr, x);
            Item it, ahead;
            auto pages = [&](const Item& i, int j) {
                const int tile = j + q;
                const bool shared = M && tile < i.pt;            // the prefix's tiles come first
                const int key = (shared || !M ? tile : tile - i.pt) * kN + (part << part_log2);
                if (part >= parts || tile >= i.j1 || key >= (shared ? a.prefix_len : i.nkeys)) return -1;
                const int p = (shared ? a.prefix_table : i.tab)[key >> a.ps_log2];
                return p >= 0 && p < a.P ? p : -1;
            };
            uint32_t n = 0;
            bool ok = true, more = false, more_next = true;
            int j = 0, val = -1, j_next = 0, val_next = -1;
            ahead.j0 = ahead.j1 = 0;
            for (int turn = 0; ok; ++turn) {
                const bool hand_on = turn == 1 || turn > 2;
                if (hand_on) {
                    it = ahead;
                    more = more_next;
                    j = j_next;
                    val = val_next;
                }
                if (more_next && turn != 1) {
                    j_next += 4;
                    if (j_next >= ahead.j1) {
                        more_next = walk.next(a, t, ahead);
                        j_next = ahead.j0;
                    }
                    val_next = more_next ? pages(ahead, j_next) : -1;
                }
                if (!hand_on) continue;
                const int last = more ? min(j + 4, it.j1) : j + 1;
                for (int jj = j; jj < last && ok; ++jj, ++n) {
                    if (!(ok = pf_wait(&sh.d_empty[x][n % kDesc], ((n / kDesc) & 1) ^ 1, wc, kPfDescEmpty))) break;
                    Desc& d = sh.desc[x][n % kDesc];
                    const uint32_t live = __ballot_sync(0xffffffffu, val >= 0);
                    if (q == jj - j) d.page[part] = val;
                    if (lane == 0) {
                        const int bits = (live >> (8 * (jj - j))) & 0xff;
                        const bool shared = M && jj < it.pt;
                        const int jt = shared || !M ? jj : jj - it.pt, nkeys = shared ? a.prefix_len : it.nkeys;
                        d.flags = more ? kMore | (jj == it.j0 ? kFirst : 0) | (jj == it.j1 - 1 ? kLast : 0) | (M && it.whole ? kWhole : 0) |
                                         ((jt + 1) * kN > nkeys || bits != (1 << parts) - 1 ? kRagged : 0) : 0;
                        d.live = bits;
                        d.j = jt;
                        d.nkeys = nkeys;
                        d.lim0 = shared ? INT_MAX / 2 : it.lim0;
                        d.hk = it.hk;
                        d.tok0 = it.tok0;
                        d.ntok = it.ntok;
                        d.seg = it.seg;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.d_full[x][n % kDesc]);
                }
                if (!more) break;
            }
            __syncwarp();
        }
    } else {
        regs_inc<208>();
        // ------------------------------------------------------------- softmax
        const int wg = warp >> 2, x = two ? 0 : wg;           // worker
        const int r = (warp & 3) * 32 + lane;                 // row of the tile == TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tO = lanes + wg * G::kColO1;
        const int tok = r / a.G + (two ? wg * a.tq : 0);      // token of the block
        const float scale = a.scale_log2;
        if (kStreams == 1 && wg == 1) {
            // d = 256 has one worker: these warps bring every item's Q into tensor
            // memory, a row a thread.  The loads run while the products of the item
            // before do; the stores wait for its last S.
            Walk<D, M> walk;
            walk.start(a, t, hdr, 0);
            Item it;
            for (uint32_t i = 0; walk.next(a, t, it); ++i) {
                uint32_t v[D / 64][32];
                const bool real = r < a.tq * a.G && tok < it.ntok;
                const uint4* src = reinterpret_cast<const uint4*>(a.q + (long long)(it.tok0 + tok) * a.q_stride + (it.hk * a.G + r - tok * a.G) * D);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    v[c / 8][c % 8 * 4] = x.x;
                    v[c / 8][c % 8 * 4 + 1] = x.y;
                    v[c / 8][c % 8 * 4 + 2] = x.z;
                    v[c / 8][c % 8 * 4 + 3] = x.w;
                }
                if (i > 0 && !pf_wait(&sh.q_empty[0], (i - 1) & 1, wc, kPfQEmpty)) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < D / 64; ++b) tmem_st32(lanes + G::kColQ + 32 * b, v[b]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_ready);
            }
            __syncwarp();
        }
        uint32_t items = 0;
        bool ok = true, valid = false, live_warp = false;
        int seg = 0, tok0 = 0, head0 = 0, lim_row = 0;
        float m_ref = -INFINITY, l = 0.f;
        for (uint32_t n = 0; x < workers; ++n) {
            if (!(ok = desc_wait(x, n))) break;
            const Desc& d = sh.desc[x][n % kDesc];
            const int flags = d.flags, live = d.live, k0 = d.j * kN;
            if (!(flags & kMore)) break;
            if (M || (flags & kFirst)) lim_row = min(d.nkeys, d.lim0 + tok);
            if (flags & kFirst) {
                valid = r < a.tq * a.G && tok < d.ntok;
                live_warp = __any_sync(0xffffffffu, valid);
                seg = d.seg;
                tok0 = d.tok0;
                head0 = d.hk * a.G;
                m_ref = -INFINITY;
                l = 0.f;
            }
            const int buf = kStreams == 2 ? wg : n & 1;
            const uint32_t tS = lanes + G::kColS + buf * G::kColSStep;
            if (!(ok = pf_wait(&sh.s_full[buf], (kStreams == 2 ? n : n >> 1) & 1, wc, kPfS))) break;
            tc_fence_after();
            if (live_warp) {
                float s[kN];
                {
                    uint32_t* su = reinterpret_cast<uint32_t*>(s);
#pragma unroll
                    for (int c = 0; c < kN; c += 32) tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(su + c));
                    tmem_wait_ld();
                }
                if (__any_sync(0xffffffffu, k0 + kN > lim_row)) {
                    const int lim = lim_row - k0;
#pragma unroll
                    for (int c = 0; c < kN; ++c)
                        if (c >= lim) s[c] = -INFINITY;
                }
                if (live != (1 << parts) - 1) {
                    // Keys of absent pages, 32 at a time (a part is a multiple of 16).
#pragma unroll
                    for (int c0 = 0; c0 < kN; c0 += 32) {
                        uint32_t w = 0;
                        for (int h = 0; h < 2; ++h)
                            if ((live >> ((c0 + 16 * h) >> part_log2)) & 1) w |= 0xffffu << (16 * h);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!((w >> c) & 1u)) s[c0 + c] = -INFINITY;
                    }
                }
                // Row maximum in four chains of three-input maxima, the
                // exponents two at a time, the row sum in two packed sums (as in
                // the forward kernels).
                float mx0 = fmaxf(s[0], s[1]), mx1 = fmaxf(s[2], s[3]), mx2 = fmaxf(s[4], s[5]), mx3 = fmaxf(s[6], s[7]);
#pragma unroll
                for (int c = 8; c < kN; c += 8) {
                    mx0 = fmax3(mx0, s[c], s[c + 1]);
                    mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
                    mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
                    mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
                }
                const float m_new = fmaxf(m_ref, fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * scale);
                // Rows that hold no query must not decide: what they hold is left over.
                const bool jump = valid && ((m_ref == -INFINITY) ? (m_new != -INFINITY) : (m_new - m_ref > kTau));
                if (__any_sync(0xffffffffu, jump)) {
                    const float fac = (m_ref == -INFINITY) ? 0.f : ex2_mufu(m_ref - m_new);
                    l *= fac;
                    if (!(flags & kFirst)) {
                        // Single-buffered S: it was issued after the worker's last
                        // P V.  Double-buffered: the P V of the tile before may
                        // still run; its barrier (of two, by turns) has completed
                        // every earlier phase, since this S was issued after the
                        // P V of two tiles before, and cannot be a phase further.
                        if (kStreams == 1) {
                            if (!(ok = pf_wait(&sh.pv_done[buf ^ 1], ((n - 1) >> 1) & 1, wc, kPfPV))) break;
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac);
                            tmem_st32(tO + c0, o);
                        }
                    }
                    m_ref = m_new;
                }
                const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
                const uint64_t sc2 = f2_pack(scale, scale), nm2 = f2_pack(-m_use, -m_use);
                uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll
                for (int st = 0; st < kN / 32; ++st) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = st * 32 + 2 * i;
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(s[c], s[c + 1]), sc2, nm2), x0, x1);
                        const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
                        if (i & 1) lb = f2_add(lb, f2_pack(p0, p1));
                        else la = f2_add(la, f2_pack(p0, p1));
                        pk[i] = pack_bf16x2(p0, p1);   // 16-bit weights feed the tensor core; l keeps 32 bits
                    }
                    tmem_st16(tS + st * 16, pk);
                }
                float a0, a1, b0, b1;
                f2_unpack(la, a0, a1);
                f2_unpack(lb, b0, b1);
                l += (a0 + a1) + (b0 + b1);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_ready[buf]);
            if (!(flags & kLast)) continue;
            // Epilogue: the rows' (m, l, O) into the segment's place.  The next
            // item's first P V overwrites O only after this warp's next P.
            if (!(ok = pf_wait(&sh.o_done[wg], items & 1, wc, kPfO))) break;
            ++items;
            tc_fence_after();
            if (M && live_warp && (flags & kWhole)) {
                // Nothing else joins: the output itself.
                const float inv = l == 0.f ? 0.f : 1.f / l;   // a NaN stays one
                const int head = head0 + r - r / a.G * a.G;
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + ((long long)(tok0 + tok) * a.Hq + head) * D);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c0, o);
                    tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float* f = reinterpret_cast<const float*>(o + 8 * q);
                            // A row that saw no key holds whatever P 0 V gave: 0.
                            dst[c0 / 8 + q] = l == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                                                       : make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                                                                    pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv));
                        }
                    }
                }
                if (valid) a.lse[(long long)head * a.T + tok0 + tok] = l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * 0.69314718055994531f;
            } else if (live_warp) {
                const long long at = (long long)seg * (pre ? a.rows_p : a.rows_s) + (two ? wg * a.tq * a.G + r : r);
                float* orow = (pre ? a.o_p : a.o_s) + at * D;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c0, o);
                    tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                         ::"l"(orow + c0 + 8 * q), "r"(o[8 * q]), "r"(o[8 * q + 1]), "r"(o[8 * q + 2]),
                                           "r"(o[8 * q + 3]), "r"(o[8 * q + 4]), "r"(o[8 * q + 5]), "r"(o[8 * q + 6]),
                                           "r"(o[8 * q + 7]) : "memory");
                    }
                }
                if (valid) (pre ? a.ml_p : a.ml_s)[at] = make_float2(m_ref, l);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sh.abort_flag != 0 && atomicCAS(&a.status->code, 0, kStatusTimeout) == 0) {
        a.status->where = sh.abort_flag;
        a.status->block = blockIdx.x;
    }
    if (warp == kSoftWarps + 3) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- join

// Bound by latency (header, row, places, (m, l), O: five loads that depend on
// one another, 3.4 us for one row, 7 from cold caches) and, with many rows, by the segments' traffic
// (512 rows of 32 heads: 23 us from a cold L2, a seventh of that out of it).
// A warp joins kHeads heads of one key/value head in one row of q: their
// segments are the same, their rows in a segment neighbours, so one set of
// places serves all and their loads overlap (many rows: 4 or 2 where they divide
// the group).  kSplit: the eight warps of a block share one head's segments
// (few rows, where a warp each would leave most SMs idle).  kRows > 1: calls whose
// items may have written their rows already.  A warp looks at so many rows, a lane
// each, and the block's warps share what there is to join.  Six prompts of up to
// 2048 tokens over 8192 shared keys, the whole call: 1113 us with a row a warp,
// 1070 on the same box with four (or eight: but four prompts without a prefix 110, 101 and 118).
template <int D, int kHeads, bool kSplit, int kRows>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PfArgs a) {
    constexpr int E = D / 32, H = kHeads;
    static_assert((!kSplit || H == 1) && (!kSplit || kRows == 1), "one head and row a block");
    __shared__ float s_o[kSplit ? 8 : 1][kSplit ? D : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = a.Hq / H;
    const long long w = kSplit ? blockIdx.x : blockIdx.x * 8LL + warp;
    const int t0 = (int)(w / groups) * kRows;
    int h0 = (int)(w % groups) * H, hk = h0 / a.G;
    if (kRows == 1 && t0 >= a.T) return;
    grid_wait();
    const PfHeader h = *a.hdr;
    if (h.bad) return;
    // Most segments that an item of the prefix can have.
    const int most = h.chunk > h.per_p ? (h.chunk - 1) / h.per_p + 2 : 2;
    PfRow r;
    int i, rb, blk, slots, tiles, units, item, u0, c_own, all;   // slots: room for all chunks' segments
    // What there is to join for row t; false: nothing, or it is written already.
    auto look = [&](int t) -> bool {
        r = a.rows[t];
        if (r.n == 0) return false;
        i = t - r.c0;
        const int nb = cdiv(r.n, a.tb);
        rb = i / a.tb;
        blk = r.block;
        slots = blk >= 0 ? most * h.chunks : 0;
        // The request's item: its units from u0 on, the workers that they fall to.
        units = units_of<true>(a, r.n, r.s);
        const int seen = r.s - r.n + min(r.n, (rb + 1) * a.tb);
        tiles = prefix_tiles<true>(a, r.n) + (seen > 0 ? (seen + (1 << a.ulog_s) - 1) >> a.ulog_s : 0);
        item = hk * nb + index_of(rb, nb);
        u0 = r.pref + item * units;
        c_own = u0 / h.per_s;
        all = slots + (tiles > 0 ? (u0 + units - 1) / h.per_s - c_own + 1 : 0);
        if (a.direct && slots == 0 && tiles > 0) {
            // Written already if one worker had all its tiles: the first that had any.
            for (int c = c_own;; ++c) {
                const int to = tile_of(min(units, c * h.per_s + h.per_s - u0), units, tiles);
                if (to == tiles && tile_of(max(0, c * h.per_s - u0), units, tiles) == 0) return false;
                if (to > 0) break;
            }
        }
        return true;
    };
    __shared__ int s_count[8], s_task[kRows > 1 ? 64 : 1][2];
    int tasks = 1;
    if constexpr (kRows > 1) {
        static_assert(kRows <= 8, "room for the tasks");
        const uint32_t todo = __ballot_sync(0xffffffffu, lane < kRows && t0 + lane < a.T && look(t0 + lane));
        if (lane == 0) s_count[warp] = __popc(todo);
        __syncthreads();
        tasks = 0;
        int at = __popc(todo & ((1u << lane) - 1u));
        for (int y = 0; y < 8; ++y) {
            if (y < warp) at += s_count[y];
            tasks += s_count[y];
        }
        if (todo >> lane & 1) {
            s_task[at][0] = t0 + lane;
            s_task[at][1] = h0;
        }
        __syncthreads();
    }
    for (int task = kRows > 1 ? warp : 0; task < tasks; task += 8) {
        const int t = kRows > 1 ? s_task[task][0] : t0;
        if (kRows > 1) {
            h0 = s_task[task][1];
            hk = h0 / a.G;
        }
        const int g0 = h0 - hk * a.G;
        if (!look(t)) return;
        // Row (of head h0) in the k-th segment, the prefix's first, then the
        // request's, each in the list's order; negative: there is none.
        auto place = [&](int k) -> long long {
            if (k >= all) return -1;
            if (k < slots) {
                const int ch = k / most, j = k - ch * most, len = min(h.chunk, a.tiles_p - ch * h.chunk);
                const int v0 = hk * h.blocks * a.tiles_p + ch * h.chunk * h.blocks + blk * len;
                const int ca = v0 / h.per_p, cb = (v0 + len - 1) / h.per_p;
                if (ca + j > cb) return -1;
                return (long long)((hk * h.chunks + ch) * h.blocks + blk + ca + j) * a.rows_p + t % a.tb * a.G + g0;
            }
            const int c = c_own + k - slots;
            const int from = max(0, c * h.per_s - u0), to = min(units, c * h.per_s + h.per_s - u0);
            if (tile_of(from, units, tiles) >= tile_of(to, units, tiles)) return -1;
            return (long long)(r.items + item + c) * a.rows_s + (i - rb * a.tb) * a.G + g0;
        };
        float M[H], L[H], acc[H][E];
#pragma unroll
        for (int x = 0; x < H; ++x) {
            M[x] = -INFINITY;
            L[x] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[x][e] = 0.f;
        }
        // Places and (m, l) of the first 32 segments, one a lane; rarely there are more.
        float2 ml[H];
        long long at = -1;
        auto load_ml = [&](int k) {
            at = place(k);
#pragma unroll
            for (int x = 0; x < H; ++x) ml[x] = at >= 0 ? (k < slots ? a.ml_p : a.ml_s)[at + x] : make_float2(-INFINITY, 0.f);
        };
        for (int k0 = (all - 1) / 32 * 32; k0 >= 0; k0 -= 32) {
            load_ml(k0 + lane);
#pragma unroll
            for (int x = 0; x < H; ++x) M[x] = fmaxf(M[x], ml[x].x);
        }
#pragma unroll
        for (int x = 0; x < H; ++x)
            for (int o = 16; o; o >>= 1) M[x] = fmaxf(M[x], __shfl_xor_sync(0xffffffffu, M[x], o));
        for (int k0 = 0; k0 < all; k0 += 32) {
            if (k0) load_ml(k0 + lane);
            float f[H];
#pragma unroll
            for (int x = 0; x < H; ++x) {
                f[x] = ml[x].y == 0.f ? 0.f : ex2_mufu(ml[x].x - M[x]);   // a sum of 0: no key seen; a NaN stays one
                L[x] += f[x] * ml[x].y;
            }
            const int cnt = min(32, all - k0);
#pragma unroll 4
            for (int k = kSplit ? warp : 0; k < cnt; k += kSplit ? 8 : 1) {
                const long long row = __shfl_sync(0xffffffffu, at, k);
                if (row < 0) continue;
                const float* src = (k0 + k < slots ? a.o_p : a.o_s) + row * D + lane * E;
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    const float fk = __shfl_sync(0xffffffffu, f[x], k);
                    float v[E];
                    if constexpr (E == 2) {
                        const float2 q = *reinterpret_cast<const float2*>(src + x * D);
                        v[0] = q.x;
                        v[1] = q.y;
                    } else {
#pragma unroll
                        for (int e = 0; e < E; e += 4) {
                            const float4 q = *reinterpret_cast<const float4*>(src + x * D + e);
                            v[e] = q.x;
                            v[e + 1] = q.y;
                            v[e + 2] = q.z;
                            v[e + 3] = q.w;
                        }
                    }
                    // A segment in which the row saw no key has weight 0 and holds
                    // whatever its idle accumulator held.
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[x][e] = fk > 0.f ? fmaf(fk, v[e], acc[x][e]) : acc[x][e];
                }
            }
        }
#pragma unroll
        for (int x = 0; x < H; ++x)
            for (int o = 16; o; o >>= 1) L[x] += __shfl_xor_sync(0xffffffffu, L[x], o);
        if constexpr (kSplit) {
#pragma unroll
            for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[0][e];
            __syncthreads();
            if (warp) return;
#pragma unroll
            for (int e = 0; e < E; ++e)
                for (int y = 1; y < 8; ++y) acc[0][e] += s_o[y][lane * E + e];
        }
#pragma unroll
        for (int x = 0; x < H; ++x) {
            const float inv = L[x] == 0.f ? 0.f : 1.f / L[x];
            uint32_t out[E / 2];
#pragma unroll
            for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[x][e] * inv, acc[x][e + 1] * inv);
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + ((long long)t * a.Hq + h0 + x) * D) + lane * (E / 2);
            if constexpr (E == 2) *dst = out[0];
            else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
            if (lane == 0) a.lse[(long long)(h0 + x) * a.T + t] = L[x] == 0.f ? -INFINITY : (M[x] + __log2f(L[x])) * 0.69314718055994531f;
        }
    }
}

// ---------------------------------------------------------------------- host

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

struct PfLayout {
    int tq, tb, rows_p, rows_s;
    size_t rows, o_p, ml_p, o_s, ml_s, total;
};

// Workspace: header, what the rows are, the segments' rows.  The prefix's items are row
// blocks times chunks of a worker's share of tiles, so at most row blocks plus
// workers; the requests' at most T / tb + min(T, B) a key/value head.  Segments:
// items plus workers (eight a CTA with few rows, else two at most).  Counted in
// rows, and never fewer than for fewer rows a segment, so that a workspace for
// the largest step serves all.
PfLayout pf_layout(int T, int B, int Hkv, int G, int d, int max_seqlen, int sms) {
    PfLayout w;
    w.tq = 128 / G;
    w.tb = d == 256 ? w.tq : 2 * w.tq;
    w.rows_p = (T < w.tb ? T : w.tb) * G;
    w.rows_s = (max_seqlen < w.tb ? max_seqlen : w.tb) * G;
    auto workers = [&](int rows, int width) -> size_t {      // rows of `width` a CTA, eight with few rows
        const int few = few_limit(d);
        return (size_t)sms * (rows <= few ? 8 * rows : 8 * few > width * rows ? 8 * few : width * rows);
    };
    const size_t all_p = (size_t)Hkv * ((T + w.tb - 1) / w.tb) * w.rows_p + workers(w.rows_p, 4);
    const size_t all_s = (size_t)Hkv * (T / w.tb + (T < B ? T : B)) * w.rows_s + workers(w.rows_s, 2);
    w.rows = align256(sizeof(PfHeader));
    w.ml_p = align256(w.rows + (size_t)T * sizeof(PfRow));
    w.ml_s = align256(w.ml_p + all_p * 8);
    w.o_p = align256(w.ml_s + all_s * 8);
    w.o_s = align256(w.o_p + all_p * d * 4);
    w.total = align256(w.o_s + all_s * d * 4);
    return w;
}

template <int D, bool M>
int launch_prefix(const CUtensorMap& tq_p, const CUtensorMap& tq_s, const CUtensorMap& tk, const CUtensorMap& tv,
                  const CUtensorMap& tk_few, const CUtensorMap& tv_few, const PfArgs& a, int sms, int grid, cudaStream_t stream) {
    using G = Pf<D>;
    const uint32_t smem = 1024 + G::kTiles + (a.B + 1) * 12 + a.B * 4 + a.listed * 4;
    static_assert(1024 + G::kTiles + (kMaxVarlenSeqs + 1) * 12 + kMaxVarlenSeqs * 4 <= G::kMaxSmem && G::kMaxSmem + sizeof(PfShared) <= 232448, "shared memory plan");
    auto kern = prefix_kernel<D, M>;
    // Once a device: the most that any batch needs.
    static std::atomic<uint64_t> prepared{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_LAUNCH;
    if (!(prepared.load(std::memory_order_relaxed) >> dev & 1)) {
        constexpr int most = Pf<D>::kMaxSmem;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return FA_ERR_LAUNCH;
        prepared.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    if (launch_dependent(kern, grid, G::kThreads, smem, stream, tq_p, tq_s, tk, tv, tk_few, tv_few, a) != cudaSuccess) return FA_ERR_LAUNCH;
    const long long rows = (long long)a.T * a.Hq;
    // Rows (of one head): up to two an SM a block each; up to 64 an SM (one or
    // two sets of warps) a warp each; past that four or two a warp.
    auto warps = [&](int heads, int each) { return (int)(((long long)cdiv(a.T, each) * (a.Hq / heads) + 7) / 8); };
    cudaError_t e;
    // Four rows a warp where items may have written theirs (see prefix_join_kernel).
    constexpr int kEach = M ? 4 : 1;
    const bool fours = M && rows > 64LL * sms && (a.tiles_p == 0 || a.max_seqlen >= a.merge_n);
    if (rows <= 2LL * sms) e = launch_dependent(prefix_join_kernel<D, 1, true, 1>, (int)rows, 256, 0, stream, a);
    else if (rows <= 64LL * sms || (a.G % 2 && !fours)) e = launch_dependent(prefix_join_kernel<D, 1, false, 1>, warps(1, 1), 256, 0, stream, a);
    else if (a.G % 4 && !fours) e = launch_dependent(prefix_join_kernel<D, 2, false, 1>, warps(2, 1), 256, 0, stream, a);
    else if (!fours) e = launch_dependent(prefix_join_kernel<D, 4, false, 1>, warps(4, 1), 256, 0, stream, a);
    else if (a.G % 2) e = launch_dependent(prefix_join_kernel<D, 1, false, kEach>, warps(1, kEach), 256, 0, stream, a);
    else if (a.G % 4) e = launch_dependent(prefix_join_kernel<D, 2, false, kEach>, warps(2, kEach), 256, 0, stream, a);
    else e = launch_dependent(prefix_join_kernel<D, 4, false, kEach>, warps(4, kEach), 256, 0, stream, a);
    return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_prefix_workspace_size(int T, int B, int Hq, int Hkv, int d, int max_seqlen) {
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 128 || max_seqlen < 1 ||
        (d != 64 && d != 128 && d != 256) || (long long)Hq * T > 0x7fffffffLL)
        return 0;
    const int sms = fa_num_sms();
    return pf_layout(T, B, Hkv, Hq / Hkv, d, max_seqlen > T ? (T > 1 ? T : 1) : max_seqlen, sms > 0 ? sms : kMaxSMs).total;
}

int fa_prefix_fwd(const void* q, int64_t q_stride, const void* k_pages, const void* v_pages, void* o, float* lse,
                  int T, int B, int Hq, int Hkv, int d, float alpha, int num_pages, int page_size,
                  const int* block_table, int table_width, const int* kv_lens, const int* cu_seqlens, int max_seqlen,
                  const int* prefix_table, int prefix_len, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
    if (!q || !k_pages || !v_pages || !o || !lse || !block_table || !kv_lens) return FA_ERR_INVALID;
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_pages < 1 || table_width < 1 || prefix_len < 0 ||
        (prefix_len > 0 && !prefix_table) || max_seqlen < 1)
        return FA_ERR_INVALID;
    if (!(alpha > 0.0f) || !isfinite(alpha)) return FA_ERR_INVALID;
    if (!cu_seqlens && T != B) return FA_ERR_INVALID;
    if (q_stride < (long long)Hq * d) return FA_ERR_INVALID;
    const int lg = page_log2(page_size);
    if ((d != 64 && d != 128 && d != 256) || lg < 0 || Hq / Hkv > 128 || B > kMaxVarlenSeqs) return FA_ERR_UNSUPPORTED;
    const long long lim = 0x7fffffffLL;
    // Key indices, a tile and a causal limit past them included, are 32 bits wide.
    if ((long long)Hq * T > lim || (long long)B * table_width > lim || (long long)table_width * page_size > kMaxKeys ||
        (long long)num_pages * page_size * Hkv > lim || prefix_len > kMaxKeys)
        return FA_ERR_UNSUPPORTED;
    if (misaligned(q, 15) || misaligned(k_pages, 15) || misaligned(v_pages, 15) || misaligned(o, 15) ||
        misaligned(lse, 15) || misaligned(block_table, 3) || misaligned(kv_lens, 3) || misaligned(cu_seqlens, 3) ||
        misaligned(prefix_table, 3) || (q_stride & 7))
        return FA_ERR_ALIGN;
    if (T == 0) return FA_OK;
    // Rows are written while others are still read.
    const size_t row = (size_t)Hq * d * 2, cache = (size_t)num_pages * Hkv * page_size * d * 2;
    const Span inputs[] = {{k_pages, cache}, {v_pages, cache}, {block_table, 4 * (size_t)B * table_width}, {kv_lens, 4 * (size_t)B},
                           {cu_seqlens, cu_seqlens ? 4 * ((size_t)B + 1) : 0},
                           {prefix_table, prefix_len > 0 ? 4 * (((size_t)prefix_len + page_size - 1) >> lg) : 0}};
    auto over_input = [&](const Span& out) {
        for (const Span& in : inputs)
            if (overlap(out, in)) return true;
        return overlap_rows(out, q, T, row, (size_t)q_stride * 2);
    };
    const Span out_o = {o, T * row}, out_lse = {lse, 4 * (size_t)Hq * T};
    if (over_input(out_o) || over_input(out_lse) || overlap(out_o, out_lse)) return FA_ERR_INVALID;
    if (max_seqlen > T) max_seqlen = T;
    const int sms = fa_num_sms();
    DevStatus* status = device_status_ptr();
    if (sms < 1 || !status) return FA_ERR_LAUNCH;
    const int G = Hq / Hkv;
    const PfLayout w = pf_layout(T, B, Hkv, G, d, max_seqlen, sms);
    if (!workspace || misaligned(workspace, 255) || workspace_bytes < w.total) return FA_ERR_WORKSPACE;
    const Span scratch = {workspace, w.total};
    if (over_input(scratch) || overlap(scratch, out_o) || overlap(scratch, out_lse)) return FA_ERR_INVALID;

    const int kN = d == 256 ? 64 : 128;
    // Few rows: at d = 256 up to 16 of a request's (see few_items; two warps for 32
    // rows take 4000 cycles a unit of 64 keys, one row tile 1600), never the prefix's
    // (3 rows of 4 heads, 32768 keys: 97 us, one row tile 61); else up to 32 (1560 a
    // unit at d = 128, one row tile 2500).
    const int mode_p = d != 256 && T * (long long)G <= few_limit(d) ? kFew : d != 256 && T > w.tq ? kTwo : kOne;
    const int mode_s = max_seqlen * (long long)G <= few_limit(d) ? kFew : d != 256 && max_seqlen > w.tq ? kTwo : kOne;
    const int ulog_p = mode_p == kFew || d == 256 ? 6 : 7, ulog_s = mode_s == kFew || d == 256 ? 6 : 7;
    // The list of tiles at its longest, with room to spare in 32 bits.
    const int over_s = mode_s == kFew && d != 256 ? 1 : 2;
    const long long tiles_s = (((long long)table_width * page_size + (1 << ulog_s) - 1) >> ulog_s) + over_s;
    const long long tiles_p = ((long long)prefix_len + (1 << ulog_p) - 1) >> ulog_p;   // both units are a tile where own items take the prefix's
    const long long blocks_s = (long long)Hkv * (T / w.tb + (T < B ? T : B)), blocks_p = (long long)Hkv * ((T + w.tb - 1) / w.tb);
    if (blocks_s * (tiles_s + tiles_p) > 1 << 30 || blocks_p * tiles_p > 1 << 30) return FA_ERR_UNSUPPORTED;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PfArgs a;
    a.table = block_table;
    a.kv_lens = kv_lens;
    a.cu = cu_seqlens;
    a.prefix_table = prefix_table;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.status = status;
    a.hdr = reinterpret_cast<PfHeader*>(ws);
    a.rows = reinterpret_cast<PfRow*>(ws + w.rows);
    a.o_p = reinterpret_cast<float*>(ws + w.o_p);
    a.o_s = reinterpret_cast<float*>(ws + w.o_s);
    a.ml_p = reinterpret_cast<float2*>(ws + w.ml_p);
    a.ml_s = reinterpret_cast<float2*>(ws + w.ml_s);
    a.o = o;
    a.lse = lse;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.W = table_width;
    a.P = num_pages;
    a.ps_log2 = lg;
    a.prefix_len = prefix_len;
    a.max_seqlen = max_seqlen;
    a.tq = w.tq;
    a.tb = w.tb;
    a.rows_p = w.rows_p;
    a.rows_s = w.rows_s;
    a.tiles_p = (int)tiles_p;
    a.blocks_p = (T + w.tb - 1) / w.tb;
    a.mode_p = mode_p;
    a.mode_s = mode_s;
    a.halves_p = T * (long long)G > 16 ? 2 : 1;
    a.halves_s = max_seqlen * (long long)G > 16 ? 2 : 1;
    a.width_p = a.mode_p == kFew ? 8 / a.halves_p : a.mode_p == kOne && d != 256 ? 2 : 1;
    a.width_s = a.mode_s == kFew ? 8 / a.halves_s : a.mode_s == kOne && d != 256 ? 2 : 1;
    a.ulog_p = ulog_p;
    a.ulog_s = ulog_s;
    a.over_s = over_s;
    a.direct = mode_s == kTwo || (d == 256 && mode_s == kOne);
    // The row blocks of requests with fewer rows: each touches five at most.
    const long long listed = B * 5LL < (T + w.tb - 1) / w.tb ? B * 5LL : (T + w.tb - 1) / w.tb;
    const int tiles_bytes = d == 64 ? Pf<64>::kTiles : d == 128 ? Pf<128>::kTiles : Pf<256>::kTiles;
    const bool merge = a.direct && prefix_len > 0 && ulog_p == ulog_s &&
                       1024 + tiles_bytes + (B + 1) * 12 + B * 4 + listed * 4 <= Pf<128>::kMaxSmem;
    a.merge_n = merge ? 4 * w.tb : INT_MAX;
    a.listed = merge ? (int)listed : 0;
    const int box_p = T < w.tq ? T : w.tq, box_s = max_seqlen < w.tq ? max_seqlen : w.tq;
    a.qstep_p = (box_p * G + 7) & ~7;
    a.qstep_s = (box_s * G + 7) & ~7;
    a.scale_log2 = alpha * 1.4426950408889634f;

    CUtensorMap tq_p = {}, tq_s = {}, tk = {}, tv = {}, tk_few = {}, tv_few = {};
    // Only the maps that a mode of this call uses are encoded (each costs the
    // host a third of a microsecond).
    const bool prefix_tiles = prefix_len > 0 && mode_p != kFew, own_tiles = mode_s != kFew || d == 256;
    const long long slots = (long long)num_pages * Hkv * page_size;
    const int part = page_size < kN ? page_size : kN;
    int rc = FA_OK;
    if (d != 256 && prefix_tiles) rc = make_map_rows(&tq_p, q, d, Hq, T, q_stride, G, box_p);
    if (d != 256 && rc == FA_OK && own_tiles) rc = make_map_rows(&tq_s, q, d, Hq, T, q_stride, G, box_s);
    if (rc == FA_OK && (prefix_tiles || own_tiles)) {
        rc = make_map_pages(&tk, k_pages, d, slots, part);
        if (rc == FA_OK) rc = make_map_pages(&tv, v_pages, d, slots, part);
    }
    // Few rows: 16 keys a copy whatever the page size, all of d at once.
    if (rc == FA_OK && (mode_p == kFew || mode_s == kFew)) {
        rc = make_map_steps(&tk_few, k_pages, d, slots);
        if (rc == FA_OK) rc = make_map_steps(&tv_few, v_pages, d, slots);
    }
    if (rc != FA_OK) return rc;
    // Twice the CTAs that one unit a worker takes, up to one an SM: code that runs
    // once comes to all SMs from the same place in L2, and CTAs without work would
    // ask for it too.
    const long long need = (blocks_p * tiles_p + a.width_p - 1) / a.width_p + (blocks_s * tiles_s + a.width_s - 1) / a.width_s;
    const int grid = 2 * need + 2 < sms ? (int)(2 * need + 2) : sms;
    auto launch = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        return a.direct ? launch_prefix<D, true>(tq_p, tq_s, tk, tv, tk_few, tv_few, a, sms, grid, stream)
                        : launch_prefix<D, false>(tq_p, tq_s, tk, tv, tk_few, tv_few, a, sms, grid, stream);
    };
    if (d == 64) return launch(std::integral_constant<int, 64>{});
    if (d == 128) return launch(std::integral_constant<int, 128>{});
    return launch(std::integral_constant<int, 256>{});
}

}  // extern "C"

// fa_prefix.cu -- fa_prefix_fwd: attention of new tokens over a shared prefix
// and each request's own paged keys (sm_103a, tcgen05 / TMEM / TMA).
//
// The prefix's K and V are read once for a block of up to 256 query rows (the
// G query heads of a key/value head, times as many tokens of any requests as
// fit), a request's own K and V once for the rows of its own tokens.  Both are
// the same work on different pages, so one persistent kernel does both:
//
//   item     one row block of one key/value head against one list of pages:
//            the prefix's (rows of any requests) or a request's (its rows);
//   unit     one tile of kN keys of one item;
//   CTA      a contiguous range of the flat list of units, so the tiles, not
//            the requests, are shared out evenly whatever the lengths are; an
//            item cut by a range's end is a segment in each of its CTAs;
//   segment  leaves its rows' (m, l, O) (maximum, sum, unnormalised output) in
//            the workspace; segment ids are item + CTA, unique because every
//            step along the list raises one of the two.
//
// A second kernel joins each output row's segments: with M = max m_s,
// O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s in fp32, in the list's order, so
// the result does not depend on timing.
//
// Within a CTA (d = 64 and 128; two softmax warpgroups, loader and UMMA issuer):
//   rows > 128    two row tiles share every K/V tile (the ping-pong of
//                 fa_fwd.cu): the shape for the prefix of a large batch and for
//                 prompts, where the tensor core sets the pace;
//   rows <= 128   one row tile; the warpgroups take alternate K/V tiles with
//                 accumulators of their own, joined in the epilogue: the shape
//                 for single tokens, where the copies set the pace and two
//                 tiles in flight hide a tile's S -> P -> O latency.
// d = 256: one row tile, one warpgroup, S double-buffered, 64-key tiles (its
// accumulator takes half of tensor memory).
//
// Keys behind the end of a list and keys of absent pages are masked by
// selection, and their V rows are zeroed in shared memory before the product
// (0 * NaN would poison the sum), so the cache's leftovers never matter.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr float kTau = 8.0f;        // rescale threshold (log2 units), as in the forward kernels
constexpr int kOverheadUnits = 1;   // an item of a request counts its tiles and this (its Q load and epilogue)

template <int D> struct Pf {
    static constexpr int kStreams = D == 256 ? 1 : 2;
    static constexpr int kN = D == 256 ? 64 : 128;               // keys a tile
    static constexpr int kBoxes = D / 64;                        // 64-column boxes a row
    static constexpr uint32_t kKVBox = kN * 128u;                // bytes of a box of a K/V tile
    static constexpr uint32_t kTile = kBoxes * kKVBox;
    static constexpr uint32_t kQBox = 16384u;                    // 128 rows x 128 B
    static constexpr uint32_t kQTile = kBoxes * kQBox;
    static constexpr int kQSlots = kStreams;
    static constexpr int kRing = D == 64 ? 8 : 4;                // 128 KB of K/V tiles
    static constexpr uint32_t kTiles = kQSlots * kQTile + kRing * kTile;
    static constexpr int kThreads = kStreams * 128 + 128;
    static constexpr uint32_t kColO1 = 128, kColS = 256, kColSStep = kN;
};

// What both kernels need to know of the list of units.
struct PfTables {
    long long* pref;     // [B+1] units of requests before b (all key/value heads)
    int* items;          // [B+1] items of requests before b
    int* cu;             // [B+1] sanitised offsets
    int* len;            // [B] own keys
};

struct PfHeader {
    long long per_p, per_s;   // units a CTA: of the prefix, of the requests
    int n_p;                  // CTAs on the prefix; the rest are on the requests
    int bad;                  // a request has more rows than max_seqlen
    int pad[10];
};

struct PfArgs {
    const int *table, *kv_lens, *cu, *prefix_table;
    DevStatus* status;
    PfHeader* hdr;
    PfTables ws;              // written by CTA 0 for the joining kernel
    float *o_p, *o_s;         // segments' rows [segment][rows][D]: prefix, requests
    float2 *ml_p, *ml_s;      // their (m, l)
    void* o;
    float* lse;
    int T, B, Hq, Hkv, G, W, P, ps_log2, prefix_len, max_seqlen;
    int tq, tb;               // tokens a row tile, a row block
    int rows_p, rows_s;       // rows a segment keeps
    int tiles_p, blocks_p;    // prefix: tiles an item, row blocks
    int weight_p, weight_s;   // relative cost of a unit
    float scale_log2;
};

enum : int { kPfQEmpty = 61, kPfRingEmpty, kPfQFull, kPfRingFull, kPfP, kPfS, kPfO, kPfExchange, kPfFree, kPfPV };

// ------------------------------------------------------------------ the list

struct Item {
    const int* tab;
    int pre, hk, tok0, ntok, j0, j1, nkeys, lim0;
    int seg;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Item k of a request's row blocks: from both ends by turns, so that under the
// causal mask two neighbours cost what any other two do.
__device__ __forceinline__ int block_of(int k, int n) { return (k & 1) ? n - 1 - (k >> 1) : k >> 1; }
__device__ __forceinline__ int index_of(int rb, int n) { return rb < (n + 1) / 2 ? 2 * rb : 2 * (n - 1 - rb) + 1; }

// A CTA's walk over its range of units.
template <int kN>
struct Walk {
    long long u, end;
    int b, hk, k, cta;
    bool pre;

    __device__ __forceinline__ static int units(const PfArgs& a, const PfTables& t, int b, int& n, int& nb) {
        n = t.cu[b + 1] - t.cu[b];
        nb = cdiv(n, a.tb);
        return n > 0 && t.len[b] > 0 ? cdiv(t.len[b], kN) + kOverheadUnits : 0;
    }

    __device__ __forceinline__ void start(const PfArgs& a, const PfTables& t, const PfHeader& h) {
        const int c = blockIdx.x;
        b = hk = k = 0;
        pre = c < h.n_p;
        cta = pre ? c : c - h.n_p;
        const long long per = pre ? h.per_p : h.per_s;
        const long long all = pre ? (long long)a.Hkv * a.blocks_p * a.tiles_p : t.pref[a.B];
        u = cta * per;
        end = u + per < all ? u + per : all;
        if (h.bad || u >= end) {
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
        const int per_item = units(a, t, b, n, nb);
        const int i = (int)((u - t.pref[b]) / per_item);
        hk = i / nb;
        k = i - hk * nb;
    }

    __device__ __forceinline__ bool next(const PfArgs& a, const PfTables& t, Item& it) {
        while (u < end) {
            if (pre) {
                const int i = (int)(u / a.tiles_p);
                it.j0 = (int)(u - (long long)i * a.tiles_p);
                const long long left = end - u;
                it.j1 = left < a.tiles_p - it.j0 ? it.j0 + (int)left : a.tiles_p;
                u += it.j1 - it.j0;
                it.hk = i / a.blocks_p;
                it.tok0 = (i - it.hk * a.blocks_p) * a.tb;
                it.ntok = min(a.tb, a.T - it.tok0);
                it.nkeys = a.prefix_len;
                it.lim0 = INT_MAX / 2;
                it.tab = a.prefix_table;
                it.seg = i + cta;
                it.pre = 1;
                return true;
            }
            int n, nb;
            const int per_item = units(a, t, b, n, nb), s = t.len[b];
            const int i = hk * nb + k;
            const int first = (int)(u - (t.pref[b] + (long long)i * per_item));
            const long long left = end - u;
            const int last = left < per_item - first ? first + (int)left : per_item;
            u += last - first;
            const int i0 = block_of(k, nb) * a.tb;
            it.hk = hk;
            it.tok0 = t.cu[b] + i0;
            it.ntok = min(a.tb, n - i0);
            it.nkeys = s;
            it.lim0 = s - n + i0 + 1;
            it.tab = a.table + (long long)b * a.W;
            it.seg = t.items[b] + i + cta;
            it.pre = 0;
            it.j0 = first;
            const int seen = it.lim0 + it.ntok - 1;        // keys the block's last row sees
            it.j1 = min(last, seen > 0 ? cdiv(seen, kN) : 0);
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

// Inclusive scan of one value a thread over the block (nthreads a multiple of 32).
template <typename V, typename Op>
__device__ __forceinline__ V block_scan(V v, V* s_warp, int tid, int nthreads, Op op) {
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = op(x, v);
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = op(s_warp[w], v);
    return v;
}

struct PfShared {
    uint64_t q_full[2], q_empty[2], full[8], empty[8], s_full[2], p_ready[2], pv_done[2], o_done, x_ready, x_free, drain;
    long long scan64[12];
    int scan32[12];
    float scanf[12];
    float2 ml[2][2][128];   // by turns: the next item's exchange may begin before the slower group has read this one's
    PfHeader hdr;
    uint32_t tmem_base;
    int abort_flag;
};

// The tables of the list, by every thread of the block: offsets by the
// library's one rule (a running maximum), units and items before each request,
// and how many CTAs work on the prefix.
template <int kN>
__device__ __forceinline__ void build_tables(const PfArgs& a, const PfTables& t, PfShared& sh, int tid, int nthreads) {
    const int per = (a.B + 1 + nthreads - 1) / nthreads, i0 = tid * per;
    int run = 0;
    auto offset = [&](int i) {
        const int c = a.cu ? a.cu[i] : i;
        return c < 0 ? 0 : (c > a.T ? a.T : c);
    };
    for (int i = i0; i < min(i0 + per, a.B + 1); ++i) run = max(run, offset(i));
    // Exclusive running maximum up to this thread's entries.
    const int upto = block_scan(run, sh.scan32, tid, nthreads, [](int x, int y) { return max(x, y); });
    int before = __shfl_up_sync(0xffffffffu, upto, 1);
    if ((tid & 31) == 0) {
        before = 0;
        for (int w = 0; w < (tid >> 5); ++w) before = max(before, sh.scan32[w]);
    }
    for (int i = i0; i < min(i0 + per, a.B + 1); ++i) {
        before = max(before, offset(i));
        t.cu[i] = before;
        if (i < a.B) {
            const long long cap = (long long)a.W << a.ps_log2;
            const int s = a.kv_lens[i];
            t.len[i] = s < 0 ? 0 : (s > cap ? (int)cap : s);
        }
    }
    if (tid == 0) sh.hdr.bad = 0;
    __syncthreads();
    long long mine = 0;
    int my_items = 0;
    float cost = 0.f;
    for (int i = i0; i < min(i0 + per, a.B); ++i) {
        int n, nb;
        const int u = Walk<kN>::units(a, t, i, n, nb);
        if (n > a.max_seqlen) sh.hdr.bad = 1;
        mine += (long long)u * nb * a.Hkv;
        my_items += nb * a.Hkv;
        // What the causal mask leaves of a row block's tiles, on average.
        const float left = fminf(1.f, fmaxf(0.f, 1.f - 0.5f * n / fmaxf((float)t.len[i], 1.f)));
        cost += (float)u * nb * a.Hkv * left;
    }
    const long long upto64 = block_scan(mine, sh.scan64, tid, nthreads, [](long long x, long long y) { return x + y; });
    const int upto_items = block_scan(my_items, sh.scan32, tid, nthreads, [](int x, int y) { return x + y; });
    const float upto_cost = block_scan(cost, sh.scanf, tid, nthreads, [](float x, float y) { return x + y; });
    long long at = upto64 - mine;
    int at_items = upto_items - my_items;
    if (tid == 0) { t.pref[0] = 0; t.items[0] = 0; }
    for (int i = i0; i < min(i0 + per, a.B); ++i) {
        int n, nb;
        const int u = Walk<kN>::units(a, t, i, n, nb);
        at += (long long)u * nb * a.Hkv;
        at_items += nb * a.Hkv;
        t.pref[i + 1] = at;
        t.items[i + 1] = at_items;
    }
    if (tid == nthreads - 1) {
        const int grid = gridDim.x;
        const long long units_p = (long long)a.Hkv * a.blocks_p * a.tiles_p, units_s = upto64;
        const float cp = (float)units_p * a.weight_p, cs = upto_cost * a.weight_s;
        int np = units_p == 0 ? 0 : (units_s == 0 ? grid : (int)(grid * (cp / (cp + cs)) + 0.5f));
        if (units_p > 0 && units_s > 0) np = grid == 1 ? 1 : max(1, min(grid - 1, np));
        const int ns = max(1, grid - np);
        sh.hdr.n_p = np;
        sh.hdr.per_p = np ? (units_p + np - 1) / np : 1;
        sh.hdr.per_s = units_s ? (units_s + ns - 1) / ns : 1;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int i = tid; i <= a.B; i += nthreads) {
            a.ws.pref[i] = t.pref[i];
            a.ws.items[i] = t.items[i];
            a.ws.cu[i] = t.cu[i];
            if (i < a.B) a.ws.len[i] = t.len[i];
        }
        if (tid == 0) {
            *a.hdr = sh.hdr;
            if (sh.hdr.bad && atomicCAS(&a.status->code, 0, -1) == 0) { a.status->where = 101; a.status->block = 0; }
        }
    }
}

// Page of the i-th part of tile j (parts are whole pages, or a tile's share of
// a larger page): its id and first row, or -1 where there is none.
template <int kN>
__device__ __forceinline__ int part_page(const PfArgs& a, const Item& it, int j, int i, int part_log2) {
    const int key = j * kN + (i << part_log2);
    if (j >= it.j1 || key >= it.nkeys) return -1;
    const int p = it.tab[key >> a.ps_log2];
    return p >= 0 && p < a.P ? p : -1;
}

// ------------------------------------------------------------------ products

template <int D>
__device__ __forceinline__ void pf_issue_qk(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem) {
    using G = Pf<D>;
    constexpr uint32_t idesc = idesc_bf16_f32(128, G::kN, 0, 0);
    const uint64_t qd = sdesc_sw128(q_smem, 16, 1024), kd = sdesc_sw128(k_smem, 16, 1024);
    static_for<D / 16>([&](auto kc) {
        constexpr uint32_t k = kc;
        constexpr uint32_t ao = ((k >> 2) * G::kQBox + (k & 3) * 32) >> 4, bo = ((k >> 2) * G::kKVBox + (k & 3) * 32) >> 4;
        umma_ss_k<ao, bo>(d_tmem, qd, kd, idesc, k > 0);
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

// -------------------------------------------------------------------- kernel

template <int D>
__global__ void __launch_bounds__(Pf<D>::kThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap tq_p, const __grid_constant__ CUtensorMap tq_s,
              const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const PfArgs a) {
    using G = Pf<D>;
    constexpr int kN = G::kN, kStreams = G::kStreams, kRing = G::kRing, kBoxes = G::kBoxes;
    constexpr int kSoftWarps = 4 * kStreams, kThreads = G::kThreads;
    extern __shared__ uint8_t dsmem[];
    __shared__ PfShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(dsmem) + 1023u) & ~1023u;
    uint8_t* gbase = dsmem + (base - smem_u32(dsmem));
    const uint32_t sQ = base, sRing = base + G::kQSlots * G::kQTile;
    PfTables t;
    t.pref = reinterpret_cast<long long*>(gbase + G::kTiles);
    t.items = reinterpret_cast<int*>(t.pref + a.B + 1);
    t.cu = t.items + a.B + 1;
    t.len = t.cu + a.B + 1;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i], 4);
            mbar_init(&sh.pv_done[i], 1);
        }
        for (int i = 0; i < kRing; ++i) { mbar_init(&sh.full[i], 1); mbar_init(&sh.empty[i], 1); }
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.x_ready, kSoftWarps);
        mbar_init(&sh.x_free, kSoftWarps);
        mbar_init(&sh.drain, 1);
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kSoftWarps && lane == 0) {
        tma_prefetch_desc(&tq_p);
        tma_prefetch_desc(&tq_s);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
    }
    if (warp == 0) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    build_tables<kN>(a, t, sh, tid, kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const WaitCtx wc{&sh.abort_flag, a.status};
    const uint32_t tmem = sh.tmem_base;
    // Parts of a tile: whole pages, or one part where a page is larger.
    const int part_log2 = min(a.ps_log2, kN == 64 ? 6 : 7), parts = kN >> part_log2;
    Walk<kN> walk;
    walk.start(a, t, sh.hdr);
    Item it;

    if (warp >= kSoftWarps) {
        if constexpr (kStreams == 2) regs_dec<72>();
        if (warp == kSoftWarps) {
            // ------------------------------------------------------------ loader
            // Lane i * kBoxes + c copies box c of part i (at most 16 lanes).
            uint32_t n_ring = 0, qc[2] = {0, 0}, qsel = 0;
            const int part = lane / kBoxes, col = lane % kBoxes;
            const bool mine = part < parts;
            const uint32_t part_bytes = 128u << part_log2;
            bool ok = true;
            auto page = [&](int j) { return mine ? part_page<kN>(a, it, j, part, part_log2) : -1; };
            auto load = [&](const CUtensorMap* map, int j, int pg) -> bool {
                const uint32_t slot = n_ring % kRing;
                if (!mbar_wait_w(&sh.empty[slot], ((n_ring / kRing) & 1) ^ 1, wc, kPfRingEmpty)) return false;
                const uint32_t live = __ballot_sync(0xffffffffu, pg >= 0);
                if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], __popc(live) * part_bytes);
                __syncwarp();
                if (pg >= 0) {
                    const int row = ((pg * a.Hkv + it.hk) << a.ps_log2) + ((j * kN + (part << part_log2)) & ((1 << a.ps_log2) - 1));
                    tma_load_2d(sRing + slot * G::kTile + col * G::kKVBox + part * part_bytes, map, &sh.full[slot], col * 64, row);
                }
                ++n_ring;
                return true;
            };
            while (ok && walk.next(a, t, it)) {
                const bool two = it.ntok > a.tq;
                const int ahead = two ? 1 : 2;
                int p0 = page(it.j0), p1 = page(it.j0 + 1), p2 = page(it.j0 + 2);
                if (!(ok = load(&tk, it.j0, p0))) break;
                // Q: one box column a lane.
                for (int x = 0; x < (two ? 2 : 1) && ok; ++x) {
                    const uint32_t qs = two ? (uint32_t)x : qsel;
                    if (!(ok = mbar_wait_w(&sh.q_empty[qs], (qc[qs] & 1) ^ 1, wc, kPfQEmpty))) break;
                    const uint32_t box = 128u * a.G * (it.pre ? a.tq : min(a.tq, a.max_seqlen));
                    if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[qs], kBoxes * box);
                    __syncwarp();
                    if (lane < kBoxes)
                        tma_load_3d(sQ + qs * G::kQTile + lane * G::kQBox, it.pre ? &tq_p : &tq_s, &sh.q_full[qs], lane * 64,
                                    it.hk * a.G, it.tok0 + x * a.tq);
                    ++qc[qs];
                }
                if (!two) qsel ^= G::kQSlots - 1;
                if (!ok) break;
                if (ahead == 2 && it.j0 + 1 < it.j1 && !(ok = load(&tk, it.j0 + 1, p1))) break;
                for (int j = it.j0; j < it.j1; ++j) {
                    const int p3 = page(j + 3);
                    if (!(ok = load(&tv, j, p0))) break;
                    if (j + ahead < it.j1 && !(ok = load(&tk, j + ahead, two ? p1 : p2))) break;
                    p0 = p1;
                    p1 = p2;
                    p2 = p3;
                }
            }
            // Every copy lands before teardown.
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t i = n_ring > kRing ? n_ring - kRing : 0; i < n_ring; ++i)
                while (!mbar_try_wait(smem_u32(&sh.full[i % kRing]), (i / kRing) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            for (int x = 0; x < G::kQSlots; ++x)
                if (qc[x] > 0)
                    while (!mbar_try_wait(smem_u32(&sh.q_full[x]), (qc[x] - 1) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            __syncwarp();
        } else if (warp == kSoftWarps + 1) {
            // ------------------------------------------------------- UMMA issuer
            uint32_t n_ring = 0, qc[2] = {0, 0}, pc[2] = {0, 0}, qsel = 0, done = 0;
            bool ok = true;
            auto col_s = [&](int x) { return tmem + G::kColS + x * G::kColSStep; };
            // Waits for the next tile of the ring; its address.
            auto take = [&](uint32_t& slot) -> bool {
                slot = n_ring % kRing;
                if (!mbar_wait_w(&sh.full[slot], (n_ring / kRing) & 1, wc, kPfRingFull)) return false;
                ++n_ring;
                return true;
            };
            // Zeroes the V rows of tile j that hold no visible key of the list
            // (live: its parts that have a page).
            auto clean = [&](uint32_t slot, int j, uint32_t live) {
                const int rows = it.nkeys - j * kN;     // of the tile's kN
                const uint32_t all = (1u << parts) - 1u;
                if (rows >= kN && live == all) return;
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
            auto live_of = [&](int j) {
                return __ballot_sync(0xffffffffu, lane < parts && part_page<kN>(a, it, j, lane, part_log2) >= 0);
            };
            while (ok && walk.next(a, t, it)) {
                const bool two = it.ntok > a.tq;
                const int n = it.j1 - it.j0;
                uint32_t ks, vs;
                uint32_t live = live_of(it.j0);
                if (two) {
                    if constexpr (kStreams == 2) {
                        if (!(ok = mbar_wait_w(&sh.q_full[0], qc[0] & 1, wc, kPfQFull))) break;
                        if (!(ok = mbar_wait_w(&sh.q_full[1], qc[1] & 1, wc, kPfQFull))) break;
                        ++qc[0];
                        ++qc[1];
                        if (!(ok = take(ks))) break;
                        tc_fence_after();
                        for (int x = 0; x < 2; ++x) {
                            pf_issue_qk<D>(col_s(x), sQ + x * G::kQTile, sRing + ks * G::kTile);
                            umma_commit_w(&sh.s_full[x]);
                        }
                        umma_commit_w(&sh.empty[ks]);
                        if (n == 1) { umma_commit_w(&sh.q_empty[0]); umma_commit_w(&sh.q_empty[1]); }
                        for (int g = 0; g < n; ++g) {
                            const bool more = g + 1 < n;
                            if (!(ok = take(vs))) break;
                            if (more && !(ok = take(ks))) break;
                            clean(vs, it.j0 + g, live);
                            live = live_of(it.j0 + g + 1);
                            if (g == 0 && done > 0 && !(ok = mbar_wait_w(&sh.x_free, (done - 1) & 1, wc, kPfFree))) break;
                            for (int x = 0; x < 2; ++x) {
                                if (!(ok = mbar_wait_w(&sh.p_ready[x], pc[x] & 1, wc, kPfP))) break;
                                ++pc[x];
                                tc_fence_after();
                                pf_issue_pv<D>(tmem + x * G::kColO1, col_s(x), sRing + vs * G::kTile, g > 0);
                                if (x == 1) umma_commit_w(&sh.empty[vs]);
                                if (more) {
                                    pf_issue_qk<D>(col_s(x), sQ + x * G::kQTile, sRing + ks * G::kTile);
                                    umma_commit_w(&sh.s_full[x]);
                                    if (g + 2 == n) umma_commit_w(&sh.q_empty[x]);
                                    if (x == 1) umma_commit_w(&sh.empty[ks]);
                                }
                            }
                            if (!ok) break;
                        }
                    }
                } else {
                    const uint32_t qs = qsel;
                    qsel ^= G::kQSlots - 1;
                    if (!(ok = mbar_wait_w(&sh.q_full[qs], qc[qs] & 1, wc, kPfQFull))) break;
                    ++qc[qs];
                    auto qk = [&](int g) {
                        pf_issue_qk<D>(col_s(g & 1), sQ + qs * G::kQTile, sRing + ks * G::kTile);
                        umma_commit_w(&sh.s_full[g & 1]);
                        umma_commit_w(&sh.empty[ks]);
                        if (g == n - 1) umma_commit_w(&sh.q_empty[qs]);
                    };
                    for (int g = 0; g < 2 && g < n; ++g) {
                        if (!(ok = take(ks))) break;
                        tc_fence_after();
                        qk(g);
                    }
                    for (int g = 0; g < n && ok; ++g) {
                        const int x = g & 1;
                        if (!(ok = take(vs))) break;
                        clean(vs, it.j0 + g, live);
                        live = live_of(it.j0 + g + 1);
                        if (g == 0 && done > 0 && !(ok = mbar_wait_w(&sh.x_free, (done - 1) & 1, wc, kPfFree))) break;
                        if (!(ok = mbar_wait_w(&sh.p_ready[x], pc[x] & 1, wc, kPfP))) break;
                        ++pc[x];
                        tc_fence_after();
                        pf_issue_pv<D>(tmem + (kStreams == 2 ? x * G::kColO1 : 0), col_s(x), sRing + vs * G::kTile, g >= kStreams);
                        umma_commit_w(&sh.empty[vs]);
                        if (kStreams == 1) umma_commit_w(&sh.pv_done[x]);
                        if (g + 2 < n) {
                            if (!(ok = take(ks))) break;
                            qk(g + 2);
                        }
                    }
                }
                if (!ok) break;
                umma_commit_w(&sh.o_done);
                ++done;
            }
            // All products complete before tensor memory is freed.
            umma_commit_w(&sh.drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&sh.drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            __syncwarp();
        }
    } else {
        if constexpr (kStreams == 2) regs_inc<216>();
        // ------------------------------------------------------------- softmax
        const int wg = warp >> 2;
        const int r = (warp & 3) * 32 + lane;                 // row of the tile == TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int r_tok = r / a.G;                            // token of the tile
        const float scale = a.scale_log2;
        uint32_t sc[2] = {0, 0}, done = 0, xc = 0;
        bool ok = true;
        auto page_bits = [&](int j) {
            return __ballot_sync(0xffffffffu, lane < parts && part_page<kN>(a, it, j, lane, part_log2) >= 0);
        };
        while (ok && walk.next(a, t, it)) {
            const bool two = it.ntok > a.tq;
            const int tok = r_tok + (two ? wg * a.tq : 0);     // token of the block
            const bool valid = r < a.tq * a.G && tok < it.ntok;
            const bool live_warp = __any_sync(0xffffffffu, valid);
            const int lim_row = it.pre ? it.nkeys : min(it.nkeys, it.lim0 + tok);
            const int step = two || kStreams == 1 ? 1 : 2;
            float m_ref = -INFINITY, l = 0.f;
            bool first = true;
            int j = it.j0 + (step == 2 ? wg : 0);
            uint32_t bits = j < it.j1 ? page_bits(j) : 0;
            for (; j < it.j1; j += step) {
                const int x = kStreams == 2 ? wg : (j - it.j0) & 1;
                const uint32_t tS = lanes + G::kColS + x * G::kColSStep;
                const uint32_t cur = bits;
                if (j + step < it.j1) bits = page_bits(j + step);
                if (!(ok = mbar_wait_w(&sh.s_full[x], sc[x] & 1, wc, kPfS))) break;
                ++sc[x];
                tc_fence_after();
                if (live_warp) {
                    float s[kN];
                    {
                        uint32_t* su = reinterpret_cast<uint32_t*>(s);
#pragma unroll
                        for (int c = 0; c < kN; c += 32) tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(su + c));
                        tmem_wait_ld();
                    }
                    const int k0 = j * kN;
                    if (__any_sync(0xffffffffu, k0 + kN > lim_row)) {
                        const int lim = lim_row - k0;
#pragma unroll
                        for (int c = 0; c < kN; ++c)
                            if (c >= lim) s[c] = -INFINITY;
                    }
                    if (cur != (1u << parts) - 1u) {
#pragma unroll
                        for (int c = 0; c < kN; ++c)
                            if (!((cur >> (c >> part_log2)) & 1u)) s[c] = -INFINITY;
                    }
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
                        if (!first) {
                            // Two streams: S of this tile was issued after the
                            // stream's last P V.  One stream: the P V of the
                            // tile before may still run; its barrier (of two,
                            // by turns) cannot be a phase further.
                            const uint32_t tO = lanes + (kStreams == 2 ? wg * G::kColO1 : 0);
                            if (kStreams == 1) {
                                if (!(ok = mbar_wait_w(&sh.pv_done[x ^ 1], (sc[x ^ 1] - 1) & 1, wc, kPfPV))) break;
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
                first = false;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_ready[x]);
            }
            if (!ok) break;
            // -------------------------------------------------------- epilogue
            // The rows' (m, l, O) into the segment's place.
            const int row = two ? wg * a.tq * a.G + r : r;
            const long long at = (long long)it.seg * (it.pre ? a.rows_p : a.rows_s) + row;
            float* orow = (it.pre ? a.o_p : a.o_s) + at * D;
            float2* ml = (it.pre ? a.ml_p : a.ml_s) + at;
            const bool join = kStreams == 2 && !two;
            float f_own = 1.f, f_other = 0.f, m = m_ref, l_all = l;
            bool other = false;
            if (join) {
                // One row tile, two streams: weights of both accumulators.
                sh.ml[xc & 1][wg][r] = make_float2(m_ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.x_ready);
                if (!(ok = mbar_wait_w(&sh.x_ready, xc & 1, wc, kPfExchange))) break;
                const float2 o2 = sh.ml[xc & 1][wg ^ 1][r];
                ++xc;
                m = fmaxf(m_ref, o2.x);
                f_own = m_ref == -INFINITY ? 0.f : ex2_mufu(m_ref - m);
                f_other = o2.x == -INFINITY ? 0.f : ex2_mufu(o2.x - m);
                l_all = l * f_own + o2.y * f_other;
                other = it.j1 - it.j0 > 1;     // the second stream had a tile
            }
            if (!(ok = mbar_wait_w(&sh.o_done, done & 1, wc, kPfO))) break;
            ++done;
            tc_fence_after();
            if (live_warp) {
                const int c_lo = join ? wg * (D / 2) : 0, c_hi = join ? c_lo + D / 2 : D;
                const uint32_t t_own = lanes + (kStreams == 2 ? (join ? 0 : wg * G::kColO1) : 0);
                const float f0 = join ? (wg == 0 ? f_own : f_other) : 1.f, f1 = wg == 0 ? f_other : f_own;
#pragma unroll 1
                for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(t_own + c0, o);
                    tmem_wait_ld();
                    if (join) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
                        if (other) {
                            uint32_t o1[32];
                            tmem_ld32(lanes + G::kColO1 + c0, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(o[i])));
                        }
                    }
                    if (valid) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                         ::"l"(orow + c0 + 8 * q), "r"(o[8 * q]), "r"(o[8 * q + 1]), "r"(o[8 * q + 2]),
                                           "r"(o[8 * q + 3]), "r"(o[8 * q + 4]), "r"(o[8 * q + 5]), "r"(o[8 * q + 6]),
                                           "r"(o[8 * q + 7]) : "memory");
                    }
                }
                if (valid && (!join || wg == 0)) *ml = make_float2(m, l_all);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.x_free);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- join

// kWarps warps a row: 1 where there are rows enough to fill the GPU, 8 (each
// takes every eighth segment) where there are few rows of many segments.
template <int D, int kWarps>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PfArgs a) {
    constexpr int kN = Pf<D>::kN, E = D / 32;
    __shared__ float s_o[kWarps == 1 ? 1 : 8][kWarps == 1 ? 1 : D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PfHeader h = *a.hdr;
    if (h.bad) return;
    const long long w = kWarps == 1 ? blockIdx.x * 8LL + warp : blockIdx.x;
    if (w >= (long long)a.T * a.Hq) return;
    const int t = (int)(w / a.Hq), head = (int)(w - (long long)t * a.Hq), hk = head / a.G, gi = head - hk * a.G;
    if (t < a.ws.cu[0] || t >= a.ws.cu[a.B]) return;
    // The request that owns row t: two rounds of 32 candidates (B <= 1024).
    int lo = 0, n_in = a.B;
    while (n_in > 1) {
        const int step = (n_in + 31) / 32, c = lo + lane * step;
        const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n_in && a.ws.cu[c] <= t);
        const int k = 31 - __clz(le);
        lo += k * step;
        n_in = min(step, n_in - k * step);
    }
    const int b = lo, c0 = a.ws.cu[b], n = a.ws.cu[b + 1] - c0, s = a.ws.len[b], i = t - c0;
    // Segments: the prefix's first, then the request's, each in the list's order.
    int np = 0, ns = 0;
    long long seg_p = 0, seg_s = 0, row_p = 0, row_s = 0;
    if (a.prefix_len > 0) {
        const int blk = t / a.tb, item = hk * a.blocks_p + blk;
        const long long u0 = (long long)item * a.tiles_p;
        const int ca = (int)(u0 / h.per_p), cb = (int)((u0 + a.tiles_p - 1) / h.per_p);
        np = cb - ca + 1;
        seg_p = item + ca;
        row_p = (t - blk * a.tb) * a.G + gi;
    }
    const int nb = cdiv(n, a.tb), rb = i / a.tb;
    const int ntok = min(a.tb, n - rb * a.tb), seen = s - n + rb * a.tb + ntok;   // of the block's last row
    if (seen > 0 && s > 0) {
        const int item = hk * nb + index_of(rb, nb);
        const long long u0 = a.ws.pref[b] + (long long)item * (cdiv(s, kN) + kOverheadUnits);
        const int ca = (int)(u0 / h.per_s), cb = (int)((u0 + cdiv(seen, kN) - 1) / h.per_s);
        ns = cb - ca + 1;
        seg_s = a.ws.items[b] + item + ca;
        row_s = (i - rb * a.tb) * a.G + gi;
    }
    const int all = np + ns;
    auto place = [&](int k) { return k < np ? (seg_p + k) * a.rows_p + row_p : (seg_s + k - np) * a.rows_s + row_s; };
    float M = -INFINITY;
    for (int k = lane; k < all; k += 32) M = fmaxf(M, (k < np ? a.ml_p : a.ml_s)[place(k)].x);
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < all; k0 += 32) {
        float f = 0.f;
        if (k0 + lane < all) {
            const float2 ml = (k0 + lane < np ? a.ml_p : a.ml_s)[place(k0 + lane)];
            f = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - M);
            L += f * ml.y;
        }
        const int cnt = min(32, all - k0);
#pragma unroll 4
        for (int k = kWarps == 1 ? 0 : warp; k < cnt; k += kWarps) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const long long at = place(k0 + k) * D + lane * E;
            const float* src = (k0 + k < np ? a.o_p : a.o_s) + at;
            float v[E];
            if constexpr (E == 2) {
                const float2 x = *reinterpret_cast<const float2*>(src);
                v[0] = x.x; v[1] = x.y;
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(src + e);
                    v[e] = x.x; v[e + 1] = x.y; v[e + 2] = x.z; v[e + 3] = x.w;
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(fk, v[e], acc[e]);
        }
    }
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if constexpr (kWarps > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int e = 0; e < E; ++e)
            for (int x = 1; x < kWarps; ++x) acc[e] += s_o[x][lane * E + e];
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t out[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + w * D) + lane * (E / 2);
    if constexpr (E == 2) *dst = out[0];
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    if (lane == 0) a.lse[(long long)head * a.T + t] = L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
}

// ---------------------------------------------------------------------- host

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

struct PfLayout {
    int tq, tb, rows_p, rows_s;
    size_t pref, items, cu, len, o_p, ml_p, o_s, ml_s, total;
};

// Workspace: header, tables, the segments' rows.  Prefix segments: one an item
// and CTA boundary; the requests': sum of ceil(n_b / tb) <= T / tb + B items a
// key/value head.
PfLayout pf_layout(int T, int B, int Hkv, int G, int d, int max_seqlen, int sms) {
    PfLayout w;
    w.tq = 128 / G;
    w.tb = d == 256 ? w.tq : 2 * w.tq;
    w.rows_p = (T < w.tb ? T : w.tb) * G;
    w.rows_s = (max_seqlen < w.tb ? max_seqlen : w.tb) * G;
    const size_t seg_p = (size_t)Hkv * ((T + w.tb - 1) / w.tb) + sms;
    const size_t seg_s = (size_t)Hkv * (T / w.tb + (T < B ? T : B)) + sms;
    w.pref = align256(sizeof(PfHeader));
    w.items = align256(w.pref + (size_t)(B + 1) * 8);
    w.cu = align256(w.items + (size_t)(B + 1) * 4);
    w.len = align256(w.cu + (size_t)(B + 1) * 4);
    w.ml_p = align256(w.len + (size_t)B * 4);
    w.ml_s = align256(w.ml_p + seg_p * w.rows_p * 8);
    w.o_p = align256(w.ml_s + seg_s * w.rows_s * 8);
    w.o_s = align256(w.o_p + seg_p * w.rows_p * d * 4);
    w.total = align256(w.o_s + seg_s * w.rows_s * d * 4);
    return w;
}

template <int D>
int launch_prefix(const CUtensorMap& tq_p, const CUtensorMap& tq_s, const CUtensorMap& tk, const CUtensorMap& tv, const PfArgs& a,
                  int sms, cudaStream_t stream) {
    using G = Pf<D>;
    const uint32_t smem = 1024 + G::kTiles + (a.B + 1) * 16 + a.B * 4;
    static_assert(1024 + G::kTiles + (kMaxVarlenSeqs + 1) * 16 + kMaxVarlenSeqs * 4 + sizeof(PfShared) <= 232448, "shared memory plan");
    auto kern = prefix_kernel<D>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return FA_ERR_LAUNCH;
    kern<<<sms, G::kThreads, smem, stream>>>(tq_p, tq_s, tk, tv, a);
    const long long rows = (long long)a.T * a.Hq;
    // Few rows: a block each (512 rows: 64 blocks of 8 rows would leave most SMs idle).
    if (rows <= 16LL * sms) prefix_join_kernel<D, 8><<<(int)rows, 256, 0, stream>>>(a);
    else prefix_join_kernel<D, 1><<<(int)((rows + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
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
    return pf_layout(T, B, Hkv, Hq / Hkv, d, max_seqlen, sms > 0 ? sms : kMaxSMs).total;
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
    if ((long long)Hq * T > lim || (long long)B * table_width > lim || (long long)table_width * page_size > lim ||
        (long long)num_pages * page_size * Hkv > lim || (long long)prefix_len + page_size > lim)
        return FA_ERR_UNSUPPORTED;
    if (misaligned(q, 15) || misaligned(k_pages, 15) || misaligned(v_pages, 15) || misaligned(o, 15) ||
        misaligned(lse, 15) || misaligned(block_table, 3) || misaligned(kv_lens, 3) || misaligned(cu_seqlens, 3) ||
        misaligned(prefix_table, 3) || (q_stride & 7))
        return FA_ERR_ALIGN;
    if (T == 0) return FA_OK;
    const int sms = fa_num_sms();
    DevStatus* status = device_status_ptr();
    if (sms < 1 || !status) return FA_ERR_LAUNCH;
    const int G = Hq / Hkv;
    const PfLayout w = pf_layout(T, B, Hkv, G, d, max_seqlen, sms);
    if (!workspace || misaligned(workspace, 255) || workspace_bytes < w.total) return FA_ERR_WORKSPACE;

    const int kN = d == 256 ? 64 : 128;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PfArgs a;
    a.table = block_table;
    a.kv_lens = kv_lens;
    a.cu = cu_seqlens;
    a.prefix_table = prefix_table;
    a.status = status;
    a.hdr = reinterpret_cast<PfHeader*>(ws);
    a.ws.pref = reinterpret_cast<long long*>(ws + w.pref);
    a.ws.items = reinterpret_cast<int*>(ws + w.items);
    a.ws.cu = reinterpret_cast<int*>(ws + w.cu);
    a.ws.len = reinterpret_cast<int*>(ws + w.len);
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
    a.tiles_p = (prefix_len + kN - 1) / kN;
    a.blocks_p = (T + w.tb - 1) / w.tb;
    a.weight_p = w.rows_p > 128 ? 2 : 1;
    a.weight_s = w.rows_s > 128 ? 2 : 1;
    a.scale_log2 = alpha * 1.4426950408889634f;

    CUtensorMap tq_p, tq_s, tk, tv;
    int rc = make_map_rows(&tq_p, q, d, Hq, T, q_stride, G, w.tq);
    if (rc == FA_OK) rc = make_map_rows(&tq_s, q, d, Hq, T, q_stride, G, max_seqlen < w.tq ? max_seqlen : w.tq);
    const long long slots = (long long)num_pages * Hkv * page_size;
    const int part = page_size < kN ? page_size : kN;
    if (rc == FA_OK) rc = make_map_pages(&tk, k_pages, d, slots, part);
    if (rc == FA_OK) rc = make_map_pages(&tv, v_pages, d, slots, part);
    if (rc != FA_OK) return rc;
    if (d == 64) return launch_prefix<64>(tq_p, tq_s, tk, tv, a, sms, stream);
    if (d == 128) return launch_prefix<128>(tq_p, tq_s, tk, tv, a, sms, stream);
    return launch_prefix<256>(tq_p, tq_s, tk, tv, a, sms, stream);
}

}  // extern "C"

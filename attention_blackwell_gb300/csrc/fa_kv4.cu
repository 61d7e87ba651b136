// fa_kv4.cu -- attention over a paged cache in 4 bits (fa_kv4_fwd) and its pages
// as bf16 (fa_kv4_expand), sm_103a.
//
// Key j has codes c and, for group g of 32 elements, a scale s_jg (fa_kv4.cuh):
//   x_j = alpha q . k_j = alpha sum_g s_jg (q_g . c_jg),
//   O = sum_j w_j v_j / sum_j w_j,  v_jg = t_jg c'_jg,  w_j = e^(x_j - M).
// Codes become fp16 by the hardware's conversion (exact).  Where rows are few they go
// from registers to the tensor core as they are: a key's scales multiply the sums of its
// groups' products, a value's scales its weight.  More rows share codes that are expanded
// and scaled in tensor and shared memory, prompts pages expanded to bf16 in the workspace.
//
// fp16 weights.  A weight times a scale spans more than fp16 does, so weights are
// kept relative to what matters for O: with key j's largest value scale in [2, 4) 2^e_j
// (below 2^-14 e_j = -15 and it is less, but 2^(e_j - 2) at least; where all its scales
// are 0, as those of a sink's value may be, e_j = -64),
//   M = max (x_j + e_j),  p_j = 2^(x_j + e_j - M + 5) in [0, 2^13],  t_jg 2^-e_j in [0, 4),
// so the largest is at least 2^6 (2^3 below 2^-14), and what falls under fp16's 2^-24 is
// 2^30 (2^27) times smaller than the largest term of O.  A key without a value holds M
// up only where it has 2^64 times another's weight.  sum_j w_j = sum_j p_j 2^-e_j stays
// in 32 bits (2^13 2^64 2^29 keys at most).  A query is scaled by a power of two into [2^14, 2^15) at its largest
// element before it becomes fp16, which all of bf16's 8 bits fit down to 2^-31 of it.
// (p is rounded to 11 bits, p t again: less than the 8 bits of a bf16 weight.)
//
// Few rows (single tokens, drafts): every warp is a worker with a range of the
// flat list of (request, key/value head, row block, 64 keys) units, a ring of
// 16-key parts in shared memory (four bulk copies a part) and its running (M, l, O) in
// registers.  Keys are the products' M, rows their N: S^T = K Q^T and O^T = V^T
// P^T, m16n8k16, so eight rows cost half of what they would as M = 16, and P goes
// from one's accumulator to the other's operand by an 8 x 8 transposition.  An item
// cut by a range's end leaves (M, l, O) in the workspace, and a second kernel joins
// the segments in the list's order; one that is not cut is written at once.
//
// More than 16 rows (8 at d = 256): a CTA is a worker, and the products
// are the fifth-generation tensor cores' (see "more rows" below): a code is converted
// once for up to 32 rows, by warps that do nothing else.
//
// Many rows (prompts): the requests' pages are expanded to bf16 once, in the
// workspace, and fa_prefix_fwd's tensor-memory pipeline does the rest: for a prompt
// the products are all, and 4.25 bits read and 16 written and read an element are
// little.
//
// What bounds it (GB300; 6.78 TB/s measured; times of calls back to back):
//   64 single tokens over up to 8191 keys each, 32 / 8 heads of 128 (303 MB): 76 us.
//   16 keys of K and V are 2176 bytes, 93 cycles of an SM's share of HBM; they take
//   290 instructions, 158 of them on the ALU (64 conversions at half rate, 16 to pair
//   value codes by keys, 20 for scales), 74 and 79 cycles of the four schedulers.
//   Measured 120: neither alone is the limit (without conversions, in an
//   experiment, 107; copies alone 93).  8 us pass before the first product: lengths,
//   walk, page numbers and copies depend on one another.  The join takes 5.
//   d = 64, 16 heads with 1 to 8 drafted tokens, up to 4096 keys (98 MB): 40 us, 186
//   instructions for 1088 bytes, the same start.
//   32 rows of 256 over up to 16384 keys (234 MB): 89 us (134 when four warps shared an
//   item's 32 rows with m16n8k16); see "more rows".
//   one token over 1017 keys: 12 to 13 us, 12 as a graph.
//   prompts, six of up to 2048 tokens over up to 10000 keys (563 GFLOP): 520 us, 25 of
//   them the expansion (164 MB), the rest fa_prefix_fwd's.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_kv4.cuh"

namespace fa {
namespace {

constexpr float kTau = 8.0f;            // rescale threshold (log2 units)
constexpr float kLift = 5.0f;           // a weight at the maximum is 2^5: 2^(kTau + kLift) times a scale below 4 fits fp16
constexpr int kQLift = 14;              // a query's largest element becomes 2^14 or more
constexpr float kNone = -3.4028234663852886e38f;   // a maximum below every finite score; a hidden key's -inf less it is -inf
constexpr int kUnit = 64;               // keys a unit
// A key's e for its value's scales, kept as e + 80: 16 (e = -64) where all are 0, else
// the largest's exponent field as an fp16 (1 to 30; e = field - 16) and 64.
constexpr uint32_t kNoValue = 16, kValue = 64;
__device__ __forceinline__ float value_e(uint32_t x) { return __uint_as_float(0x4b000000u | x) - 8388688.f; }
__device__ __forceinline__ float value_back(uint32_t x) { return __uint_as_float((207u - x) << 23); }    // 2^-e
constexpr int kMaxKeys = 1 << 29;       // of a request
constexpr int kExtraMost = 12;          // units that an item costs besides its keys', at most
constexpr int kPrefetchMost = 1 << 20;  // bytes of block tables that are brought to L2
// Rows of a request and key/value head above which pages are expanded, for all of a call's
// requests.  From the codes and expanded (us):
//   requests x keys, heads      d/2 rows    d rows     2 d rows   4 d rows
//   128: 8 x 8000, 8              72 133    128 142    239 159    462 202
//        8 x 500, 8               21  28     29  32     48  43     80  31
//        64 x 2000, 8            168 251    318 270    586 282   1162 401
//        64 x 500, 2              29  35     48  39     80  33    150  73
//        2 x 30000, 8             66 130    116 134    216 138    415 181
//        1 x 1000, 1              15  20     15  21     16  22     16  23
//    64: 8 x 8000, 8              41  71     67  89    116  97    216 115
//        64 x 2000, 8             79 130    145 170    271 189    524 186
//   256: 8 x 8000, 2              58  78     98  89    181 122    344 186
//        64 x 2000, 2            143 149    264 194    521 264    932 397
// d is nearest to where the two cross; with many requests of 128 and 256 that is about
// d/2 (at d they take up to 1.4 times as long as expanded), with one short one past 4 d.
constexpr int many_rows(int d) { return d; }
constexpr size_t kExpandMost = 4ull << 30;   // bytes of expanded pages a call takes

// A CTA's tables of the list: in shared memory up to kTableMost requests, else in its
// own piece of the workspace.
constexpr int kTableMost = 128;
__host__ __device__ constexpr uint32_t table_bytes(int B) { return (4u * B + 3) * 4; }

template <int D, int NT> struct Kv {
    static constexpr int kRows = 8 * NT, kExtra = 1;     // rows of an item
    static constexpr int kGroups = D / 32;
    static constexpr int kWorkers = D == 64 || NT * D <= 128 ? 12 : 8, kThreads = 32 * kWorkers;   // a CTA's warps, one CTA an SM
    static constexpr int kParts = D == 64 && NT == 1 ? 4 : D <= 128 ? 2 : 1;   // 16-key parts a step
    static constexpr int kSteps = D == 128 || (D == 64 && NT == 2) ? 2 : 1;   // steps a slot of the ring
    static constexpr int kSlotParts = kParts * kSteps, kKeys = 16 * kParts;
    // A slot's keys in shared memory: K's codes, V's codes, K's scales, V's scales.
    static constexpr uint32_t kCodes = 8 * D, kScales = D / 2, kPart = 2 * (kCodes + kScales), kSlot = kSlotParts * kPart;
    static constexpr uint32_t kRing = D == 128 ? (NT == 1 ? 2 : 3) : D == 64 ? (NT == 1 ? 4 : 3) : 5;
    // A step's scales as the products want them: K's as floats [key][group], V's as pairs of
    // keys [key / 2][group], (e, 2^-e) [key].
    static constexpr uint32_t kVPairs = kKeys * kGroups * 4, kExp = kVPairs + kKeys * kGroups * 2, kPrep = kExp + kKeys * 8;
    static constexpr uint32_t kWarp = kRing * kSlot + kPrep;
    static_assert(NT <= 2 && NT * D <= 256, "Q and O are in registers");
    static_assert(kPart % 16 == 0 && kWarp % 16 == 0 && kVPairs % 16 == 0 && kExp % 16 == 0 && kPrep % 16 == 0, "copies are 16-byte aligned");
    static_assert(kRing * kSlotParts <= 32 && kRing <= 8 && 4 * kSlotParts <= 32, "a bit a part, a lane a copy");
    static_assert(kWorkers * kWarp + table_bytes(kTableMost) + 1536 <= 232448, "shared memory plan");
};

struct KvRow {
    int c0, n, s, pref, items, pad[3];   // of a row's request: first row, rows (0: none), keys; units and items before it
};
struct KvHeader {
    int per, more, bad, pad;             // units a worker, the first `more` one more; a request has more rows than max_seqlen
};
// A worker's first unit, and the worker of a unit.
__device__ __forceinline__ int unit_of(const KvHeader& h, int worker) { return worker * h.per + min(worker, h.more); }
__device__ __forceinline__ int worker_of(const KvHeader& h, int unit) {
    const int longer = h.more * (h.per + 1);
    return unit < longer ? unit / (h.per + 1) : h.more + (unit - longer) / h.per;
}

struct KvArgs {
    const uint8_t *kp, *ks, *vp, *vs;
    const __nv_bfloat16* q;
    long long q_stride;
    const int *table, *kv_lens, *cu;
    __nv_bfloat16* o;
    float* lse;
    DevStatus* status;
    KvHeader* hdr;
    int* tables;             // [CTA][4 B + 3], B > kTableMost
    KvRow* rows;             // [T]
    float2* ml;              // segments' rows: maximum less kLift, sum
    float* seg;              // [segment][rows][D]
    int T, B, Hq, Hkv, G, W, P, ps_log2, max_seqlen;
    float scale_log2;
};

struct KvTables {
    int *pref, *items, *cu, *len;        // [B+1], [B+1], [B+1], [B]
};

// Row blocks of a request with n tokens, units of each of its items: its tiles of
// keys and `extra` for what an item costs besides.
// (T * Hq fits 31 bits, so rows of a request do.)
__device__ __forceinline__ int row_blocks(int n, int G, int rows) { return (int)(((uint32_t)(n * G) + (uint32_t)rows - 1) / (uint32_t)rows); }
__device__ __forceinline__ int item_units(int s, int extra) { return s > 0 ? (s + kUnit - 1) / kUnit + extra : 0; }

// The keys that row block rb's last row sees.
__device__ __forceinline__ int keys_seen(int n, int s, int G, int rb, int rows) {
    const uint32_t last = min((uint32_t)(rb + 1) * (uint32_t)rows, (uint32_t)(n * G)) - 1;
    return s - n + (int)(last / (uint32_t)G) + 1;
}

// The parts that units [first, last) of an item stand for.
__device__ __forceinline__ void parts_of(int first, int last, int seen, int extra, int& p0, int& p1) {
    p0 = max(first - extra, 0) * (kUnit / 16);
    p1 = min(max(last - extra, 0) * (kUnit / 16), seen > 0 ? (seen + 15) >> 4 : 0);
}

struct KvItem {
    int b, hk, rb, rows;     // request, key/value head, row block, its rows
    int c0, n, s;
    int p0, p1, seen;        // parts [p0, p1), keys its last row sees
    int seg;
    bool whole;              // all its parts are here
};

// A worker's walk over its units.
template <int ROWS, int EXTRA>
struct KvWalk {
    int u, end, b, worker;
    __device__ __forceinline__ void start(const KvArgs& a, const KvTables& t, const KvHeader& h, int w) {
        worker = w;
        u = h.bad ? 0 : unit_of(h, w);
        end = h.bad ? 0 : unit_of(h, w + 1);
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (t.pref[mid + 1] > u) hi = mid; else lo = mid + 1;
        }
        b = lo;
    }
    __device__ __forceinline__ bool next(const KvArgs& a, const KvTables& t, KvItem& it) {
        while (u < end) {
            while (t.pref[b + 1] <= u) ++b;
            const int n = t.cu[b + 1] - t.cu[b], s = t.len[b], per = item_units(s, EXTRA), nb = row_blocks(n, a.G, ROWS);
            const int at = u - t.pref[b], i = at / per, first = at - i * per, last = min(per, first + end - u);
            u += last - first;
            const int hk = i / nb, rb = i - hk * nb, seen = keys_seen(n, s, a.G, rb, ROWS);
            int p0, p1;
            parts_of(first, last, seen, EXTRA, p0, p1);
            if (p0 >= p1) continue;
            it.b = b;
            it.hk = hk;
            it.rb = rb;
            it.rows = min(ROWS, n * a.G - rb * ROWS);
            it.c0 = t.cu[b];
            it.n = n;
            it.s = s;
            it.p0 = p0;
            it.p1 = p1;
            it.seen = seen;
            it.seg = t.items[b] + i + worker;      // one of the two rises with every segment
            it.whole = p0 == 0 && p1 == (seen + 15) >> 4;
            return true;
        }
        return false;
    }
};

struct KvScan {
    int2 scan[28];
    int abort_flag, bad;
};
struct KvShared : KvScan {
    uint64_t full[16][8];
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// The bounded wait (2 s), by a whole warp: it looks at this CTA's flag alone, which
// takes the site that gave up, and the CTA reports it as it ends.
__device__ __forceinline__ bool kv_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const uint32_t at = smem_u32(bar);
    bool ok = mbar_try_wait(at, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (!(ok = mbar_try_wait(at, parity))) {
            if (*abort_flag) break;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// The list's tables, by every thread of the block; offsets by the library's one rule.
template <class K>
__device__ __forceinline__ KvHeader build_tables(const KvArgs& a, const KvTables& t, KvScan& sh, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    const long long cap = (long long)a.W << a.ps_log2;
    bool fine = true;
    for (int i = tid; i <= a.B; i += K::kThreads) {
        const int c = a.cu ? a.cu[i] : i, before = a.cu && i > 0 ? a.cu[i - 1] : 0;
        fine = fine && c >= before && c >= 0 && c <= a.T;
        t.cu[i] = c;
        if (i < a.B) {
            const int s = a.kv_lens[i];
            t.len[i] = s < 0 ? 0 : s > cap ? (int)cap : s;
        }
    }
    if (tid == 0) sh.bad = 0;
    if (!__syncthreads_and(fine)) {
        if (tid == 0) {      // rare, and short: at most 1025 offsets
            int run = 0;
            for (int i = 0; i <= a.B; ++i) {
                const int c = t.cu[i];
                run = max(run, c < 0 ? 0 : c > a.T ? a.T : c);
                t.cu[i] = run;
            }
        }
        __syncthreads();
    }
    int units = 0, items = 0;
    constexpr int kThreads = K::kThreads, kWarps = kThreads / 32;
    for (int base = 0; base < a.B; base += kThreads) {
        const int i = base + tid;
        int u = 0, it = 0;
        if (i < a.B) {
            const int n = t.cu[i + 1] - t.cu[i];
            if (n > a.max_seqlen) sh.bad = 1;
            it = row_blocks(n, a.G, K::kRows) * a.Hkv;
            u = it * item_units(t.len[i], K::kExtra);
        }
        const int u_own = u, it_own = it;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, u, o), y = __shfl_up_sync(0xffffffffu, it, o);
            if (lane >= o) u += x, it += y;
        }
        if (base) __syncthreads();
        if (lane == 31) sh.scan[warp] = make_int2(u, it);
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) {
            const int2 x = sh.scan[w];
            if (w < warp) u += x.x, it += x.y;
        }
        if (i < a.B) {
            t.pref[i] = units + u - u_own;
            t.items[i] = items + it - it_own;
        }
        for (int w = 0; w < kWarps; ++w) units += sh.scan[w].x, items += sh.scan[w].y;
    }
    if (tid == 0) {
        t.pref[a.B] = units;
        t.items[a.B] = items;
    }
    __syncthreads();
    KvHeader h = {};
    const int workers = gridDim.x * K::kWorkers;
    h.per = units / workers;
    h.more = units - h.per * workers;
    h.bad = sh.bad;
    if (blockIdx.x == 0 && tid == 0) {
        *a.hdr = h;
        if (h.bad && atomicCAS(&a.status->code, 0, -1) == 0) { a.status->where = 111; a.status->block = 0; }
    }
    return h;
}

// What the joining kernel needs to know of each row.
template <class K> __device__ __forceinline__ void fill_rows(const KvArgs& a, const KvTables& t, int tid) {
    for (int i = blockIdx.x * K::kThreads + tid; i < a.T; i += gridDim.x * K::kThreads) {
        KvRow row = {};
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
        }
        a.rows[i] = row;
    }
}

// Small block tables on their way to L2 while the list is made: the first lookup is
// on the way to every worker's first copy.
template <class K> __device__ __forceinline__ void prefetch_tables(const KvArgs& a, int tid) {
    const long long bytes = (long long)a.B * a.W * 4, line = ((long long)blockIdx.x * K::kThreads + tid) * 128;
    if (bytes <= kPrefetchMost && line < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(a.table) + line));
}

// ------------------------------------------------------------------ products

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// N words from or to shared memory at a 4 N-byte boundary (16 bytes at most at a time).
template <int N> __device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(p + 4 * i);
            w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
        }
    }
}
template <int N> __device__ __forceinline__ void sts(uint8_t* p, const uint32_t (&w)[N]) {
    if constexpr (N == 1) *reinterpret_cast<uint32_t*>(p) = w[0];
    else if constexpr (N == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}

// A key's scales as f16 pairs (groups 2i and 2i + 1).
template <int D> __device__ __forceinline__ void scale_pairs(const uint8_t* p, bool real, uint32_t (&h)[D / 64]) {
    uint32_t w[D == 256 ? 2 : 1];
    if constexpr (D == 64) {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
        lds(p, w);
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) h[i] = __byte_perm(real ? w[i / 2] : 0u, 0u, i & 1 ? 0x4342 : 0x4140) << 7;
}

// A step's scales, a key a lane: each is wanted by eight or four lanes, so the work is
// done once (as part of every lane's it was a quarter of all instructions).  `real`:
// this key is seen by some row; one that is not has value scales 0.
template <int D, int NT>
__device__ __forceinline__ void prepare_key(const uint8_t* ks, const uint8_t* vs, uint8_t* prep, int key, int lane, bool real) {
    using K = Kv<D, NT>;
    constexpr int kG = K::kGroups;
    uint32_t h[kG / 2], f[kG];
    scale_pairs<D>(ks + key * kG, true, h);
#pragma unroll
    for (int i = 0; i < kG / 2; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = __float_as_uint(x.x);
        f[2 * i + 1] = __float_as_uint(x.y);
    }
    sts(prep + key * (4 * kG), f);
    scale_pairs<D>(vs + key * kG, real, h);
    // 2^e from 2^-14, fp16's smallest normal number, to 2^15; a NaN counts for nothing here.
    uint32_t m = h[0];
#pragma unroll
    for (int i = 1; i < kG / 2; ++i) m = hmax2(m, h[i]);
    m = hmax2(m, __byte_perm(m, m, 0x1032));
    const uint32_t ex = hmin2(hmax2(m, 0x04000400u), 0x78007800u) & 0x7c007c00u, down = 0x7c007c00u - ex;    // 2^(16 - field) = 2^-e
#pragma unroll
    for (int i = 0; i < kG / 2; ++i) h[i] = hmul2(h[i], down);
    const uint32_t at = m ? (ex >> 26) + kValue : kNoValue;
    const uint32_t eb[2] = {__float_as_uint(value_e(at)), __float_as_uint(value_back(at))};
    sts(prep + K::kExp + key * 8, eb);
    // Pairs of keys, in the order of the products' key axis (1 0 in the second and
    // third pair of eight): the even key's lane takes the first half of the groups.
    const bool odd = lane & 1, turned = (key >> 1 ^ key >> 2) & 1;
    const uint32_t lo = turned ? 0x1054 : 0x5410, hi = turned ? 0x3276 : 0x7632;
    if constexpr (kG == 2) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, h[0], 1);
        const uint32_t out[1] = {odd ? __byte_perm(other, h[0], hi) : __byte_perm(h[0], other, lo)};
        sts(prep + K::kVPairs + (key >> 1) * 8 + (odd ? 4 : 0), out);
    } else {
        uint32_t out[kG / 2];
#pragma unroll
        for (int i = 0; i < kG / 4; ++i) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? h[i] : h[kG / 4 + i], 1);
            const uint32_t x = odd ? other : h[i], y = odd ? h[kG / 4 + i] : other;
            out[2 * i] = __byte_perm(x, y, lo);
            out[2 * i + 1] = __byte_perm(x, y, hi);
        }
        sts(prep + K::kVPairs + (key >> 1) * (4 * kG) + (odd ? 2 * kG : 0), out);
    }
}

// -------------------------------------------------------------------- kernel

template <int D, int NT>
__global__ void __launch_bounds__(Kv<D, NT>::kThreads, 1) kv4_kernel(const KvArgs a) {
    using K = Kv<D, NT>;
    constexpr int kG = K::kGroups, kParts = K::kParts, kSteps = K::kSteps, kSP = K::kSlotParts;
    constexpr uint32_t kRing = K::kRing;
    extern __shared__ __align__(16) uint8_t dsmem[];
    __shared__ KvShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    // Index i of the products' key axis is key i ^ (i >> 1) of each eight: the rows that
    // lanes read together then lie in different banks (V's loads, in order: four
    // wavefronts for one at d = 128, two at d = 64).
    const int kr = r ^ (r >> 1);
    KvTables t;
    t.pref = a.B <= kTableMost ? reinterpret_cast<int*>(dsmem + K::kWorkers * K::kWarp) : a.tables + (long long)blockIdx.x * (4 * a.B + 3);
    t.items = t.pref + a.B + 1;
    t.cu = t.items + a.B + 1;
    t.len = t.cu + a.B + 1;
    if (tid < K::kWorkers * (int)kRing) {
        mbar_init(&sh.full[tid / kRing][tid % kRing], 1);
        fence_mbar_init();
    }
    if (tid == 0) sh.abort_flag = 0;
    grid_launch_next();
    grid_wait();
    prefetch_tables<K>(a, tid);
    const KvHeader hdr = build_tables<K>(a, t, sh, tid);

    fill_rows<K>(a, t, tid);

    uint64_t* full = sh.full[warp];
    uint8_t* const ring = dsmem + warp * K::kWarp;
    uint8_t* const prep = ring + kRing * K::kSlot;
    const int worker = blockIdx.x * K::kWorkers + warp;

    // The copies: a walk of their own, ahead of the work by what the ring holds.
    KvWalk<K::kRows, K::kExtra> ahead;
    KvItem to = {};
    ahead.start(a, t, hdr, worker);
    bool more = ahead.next(a, t, to);
    int part = to.p0, win = -1, win_next = -1;       // next part; pages of its 32 parts, one a lane, and of the next 32
    uint32_t filled = 0, issued = 0, live = 0;       // next slot, slots filled, one bit a part of a slot: its page exists
    auto pages = [&](int p) -> int {                 // of parts p .. p + 31
        if (p + lane >= to.p1) return -1;
        const int x = a.table[(long long)to.b * a.W + ((p + lane) * 16 >> a.ps_log2)];
        return x >= 0 && x < a.P ? x : -1;
    };
    if (more) {
        win = pages(part);
        win_next = pages(part + 32);
    }
    // This lane's copies: one of K's codes, V's codes, K's scales and V's scales, of
    // one part of a step.
    const int what = lane & 3, which = lane >> 2;
    const uint8_t* const from = what == 0 ? a.kp : what == 1 ? a.vp : what == 2 ? a.ks : a.vs;
    const uint32_t bytes = what < 2 ? K::kCodes : K::kScales;
    const uint32_t into = smem_u32(ring) + (what < 2 ? (what * kSP + which) * K::kCodes : 2 * kSP * K::kCodes + ((what - 2) * kSP + which) * K::kScales);
    auto copy = [&]() {
        if (!more) return;
        const int page = __shfl_sync(0xffffffffu, win, (part - to.p0 + which) & 31);      // -1 past the item's end
        const bool real = lane < 4 * kSP && page >= 0;
        uint32_t on = __ballot_sync(0xffffffffu, real);
        on = kSP == 4 ? (on & 1) | (on >> 3 & 2) | (on >> 6 & 4) | (on >> 9 & 8) : kSP == 2 ? (on & 1) | (on >> 3 & 2) : on & 1;
        uint64_t* bar = &full[filled];
        __syncwarp();                                // every lane has read what the slot held
        if (lane == 0) {
            if (on) mbar_arrive_expect_tx(bar, K::kPart * __popc(on));
            else mbar_arrive(bar);
        }
        __syncwarp();
        if (real) {
            const int key = (part + which) * 16;
            const long long row = (((long long)page * a.Hkv + to.hk) << a.ps_log2) + (key & ((1 << a.ps_log2) - 1));
            bulk_load(into + filled * K::kSlot, from + row * (what < 2 ? D / 2 : D / 32), bytes, bar);
        }
        live = (live & ~(((1u << kSP) - 1u) << (filled * kSP))) | on << (filled * kSP);
        filled = filled + 1 == kRing ? 0 : filled + 1;
        ++issued;
        part += kSP;
        if (part >= to.p1) {
            more = ahead.next(a, t, to);
            if (more) {
                part = to.p0;
                win = pages(part);
                win_next = pages(part + 32);
            }
        } else if (((part - to.p0) & 31) == 0) {
            win = win_next;
            win_next = pages(part + 32);
        }
    };
    copy();

    KvWalk<K::kRows, K::kExtra> walk;
    KvItem it;
    walk.start(a, t, hdr, worker);
    uint32_t read = 0, slot = 0, phase = 0;
    bool ok = true;
    while (ok && walk.next(a, t, it)) {
        // Q as B operands: lane (r, c) has row r's elements 32 g + 8 c to + 7, which
        // are what it reads of a key.
        uint32_t qf[NT][kG][4];
        // What a row's sums are multiplied by, and the keys it sees, of rows 2c and 2c + 1.
        float f[NT][2];
        int lim[NT][2];
        float m[NT][2], l[NT][2], o[kG][2][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int x = n * 8 + r;
            const uint32_t row = (uint32_t)it.rb * K::kRows + x;
            const int tok = (int)(row / (uint32_t)a.G), h = (int)row - tok * a.G;
            uint4 in[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                in[g] = make_uint4(0, 0, 0, 0);
                if (x < it.rows)
                    in[g] = *reinterpret_cast<const uint4*>(a.q + (long long)(it.c0 + tok) * a.q_stride + (it.hk * a.G + h) * D + 32 * g + 8 * c);
            }
            float most = 0.f;
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                const uint32_t w[4] = {in[g].x, in[g].y, in[g].z, in[g].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int e = min(max((int)(__float_as_uint(most) >> 23), kQLift + 1), 254);      // exponent field: 2^(e - 127)
            const float down = __uint_as_float((uint32_t)(254 + kQLift - e) << 23), up = a.scale_log2 * __uint_as_float((uint32_t)(e - kQLift) << 23);
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                const uint32_t w[4] = {in[g].x, in[g].y, in[g].z, in[g].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[n][g][i] = pack_f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) f[n][i] = __shfl_sync(0xffffffffu, up, 8 * c + 4 * i);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tk = (int)(((uint32_t)it.rb * K::kRows + nt * 8 + 2 * c + i) / (uint32_t)a.G);
                lim[nt][i] = min(it.s, it.s - it.n + tk + 1);
                m[nt][i] = kNone;
                l[nt][i] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < kG; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[g][0][nt][i] = o[g][1][nt][i] = 0.f;
        }
        const int lim_min = it.s - it.n + (int)((uint32_t)it.rb * K::kRows / (uint32_t)a.G) + 1;

        for (int p = it.p0; p < it.p1; p += kParts) {
            const int k0 = p * 16, sub = kSteps == 1 ? 0 : (p - it.p0) / kParts & (kSteps - 1);    // step of the slot
            // The step's K codes, K scales; V's lie kSP parts behind each.
            const uint8_t* const at = ring + slot * K::kSlot + sub * (kParts * K::kCodes);
            const uint8_t* const scales = ring + slot * K::kSlot + 2 * kSP * K::kCodes + sub * (kParts * K::kScales);
            if (sub == 0) {
                ok = kv_wait(&full[slot], phase, &sh.abort_flag);
                if (!ok) break;
                // The ring is filled once the first slot is there: all at once, every
                // warp's first slot would wait for the others' second.
                if (read == 0)
                    for (uint32_t i = 1; i < kRing; ++i) copy();
            }
            const uint32_t here = live >> (slot * kSP + sub * kParts) & ((1u << kParts) - 1u);
            const bool ragged = k0 + kParts * 16 > lim_min || here != (1u << kParts) - 1u;
#pragma unroll
            for (int i = 0; i < (K::kKeys + 31) / 32; ++i) {
                const int key = i * 32 + (lane & (K::kKeys - 1));      // sixteen keys: every key twice, with the same results
                const bool real = !ragged || (k0 + key < it.seen && (here >> (key >> 4) & 1u));
                prepare_key<D, NT>(scales, scales + kSP * K::kScales, prep, key, lane, real);
            }
            __syncwarp();
            float z[kParts][NT][4], back[kParts][2];     // scores + e, 2^-e
#pragma unroll
            for (int kt = 0; kt < kParts; ++kt) {
                // Keys' codes: eight adjacent elements of every group, for keys r and r + 8.
                uint32_t kw[2][kG], ksc[2][kG];
                uint64_t z2[NT][2];                  // rows 2c and 2c + 1 of key r, of key r + 8
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds(at + (kt * 16 + kr + 8 * i) * (D / 2) + c * (D / 8), kw[i]);
                    lds(prep + (kt * 16 + kr + 8 * i) * (4 * kG), ksc[i]);
                }
#pragma unroll
                for (int j = 0; j < kG / 2; ++j) {
                    uint32_t x[2][2][4];             // [step of the group][key r, r + 8][group 2j: two pairs, group 2j + 1: two]
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        codes_f16(kw[i][j], x[0][i][0], x[0][i][1], x[0][i][2], x[0][i][3]);
                        codes_f16(kw[i][kG / 2 + j], x[1][i][0], x[1][i][1], x[1][i][2], x[1][i][3]);
                    }
#pragma unroll
                    for (int gg = 0; gg < 2; ++gg) {
                        const int g = 2 * j + gg;
                        uint64_t sc[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) sc[i] = f2_pack(__uint_as_float(ksc[i][g]), __uint_as_float(ksc[i][g]));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t (&q)[4] = qf[nt][g];
                            float acc[4];
                            mma_f16_0(acc, x[0][0][2 * gg], x[0][1][2 * gg], x[0][0][2 * gg + 1], x[0][1][2 * gg + 1], q[0], q[1]);
                            mma_f16(acc, x[1][0][2 * gg], x[1][1][2 * gg], x[1][0][2 * gg + 1], x[1][1][2 * gg + 1], q[2], q[3]);
#pragma unroll
                            for (int i = 0; i < 2; ++i) z2[nt][i] = g == 0 ? f2_mul(sc[i], f2_pack(acc[2 * i], acc[2 * i + 1])) : f2_fma(sc[i], f2_pack(acc[2 * i], acc[2 * i + 1]), z2[nt][i]);
                        }
                    }
                }
                uint32_t eb[2][2];                   // of keys r and r + 8
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds(prep + K::kExp + (kt * 16 + kr + 8 * i) * 8, eb[i]);
                    back[kt][i] = __uint_as_float(eb[i][1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e = __uint_as_float(eb[i][0]);
                        f2_unpack(f2_fma(z2[nt][i], f2_pack(f[nt][0], f[nt][1]), f2_pack(e, e)), z[kt][nt][2 * i], z[kt][nt][2 * i + 1]);
                    }
                }
            }
            if (ragged) {
#pragma unroll
                for (int kt = 0; kt < kParts; ++kt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(here >> kt & 1u) || k0 + kt * 16 + kr + (i >> 1) * 8 >= lim[nt][i & 1]) z[kt][nt][i] = -INFINITY;
            }
            // O and l follow a row's running maximum (m: kLift below it) when it grows by more
            // than kTau: only then do the lanes that share the row look for it together.
            bool jump = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(z[0][nt][i], z[0][nt][2 + i]);
#pragma unroll
                    for (int kt = 1; kt < kParts; ++kt) x = fmax3(x, z[kt][nt][i], z[kt][nt][2 + i]);
                    jump |= x - m[nt][i] > kTau + kLift;
                }
            // Weights as B operands: row r, keys 2c, 2c + 1 and eight further.
            auto weigh = [&](int kt, uint32_t (&pt)[NT][2]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
                    uint64_t sum = f2_pack(l[nt][0], l[nt][1]);
                    const uint64_t minus_m = f2_pack(-m[nt][0], -m[nt][1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f2_unpack(f2_add(f2_pack(z[kt][nt][2 * i], z[kt][nt][2 * i + 1]), minus_m), w[2 * i], w[2 * i + 1]);
                        w[2 * i] = ex2_mufu(w[2 * i]);
                        w[2 * i + 1] = ex2_mufu(w[2 * i + 1]);
                        sum = f2_fma(f2_pack(w[2 * i], w[2 * i + 1]), f2_pack(back[kt][i], back[kt][i]), sum);
                    }
                    f2_unpack(sum, l[nt][0], l[nt][1]);
                    pt[nt][0] = transposed(pack_f16x2(w[0], w[1]));
                    pt[nt][1] = transposed(pack_f16x2(w[2], w[3]));
                }
            };
            if (__any_sync(0xffffffffu, jump)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(z[0][nt][i], z[0][nt][2 + i]);
#pragma unroll
                        for (int kt = 1; kt < kParts; ++kt) x = fmax3(x, z[kt][nt][i], z[kt][nt][2 + i]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        x = fmaxf(m[nt][i], x - kLift);
                        const float fac = ex2_mufu(m[nt][i] - x);
                        l[nt][i] *= fac;
                        m[nt][i] = x;
#pragma unroll
                        for (int g = 0; g < kG; ++g)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                o[g][h][nt][i] *= fac;
                                o[g][h][nt][2 + i] *= fac;
                            }
                    }
            }
#pragma unroll
            for (int kt = 0; kt < kParts; ++kt) {
                uint32_t pt[NT][2];
                const uint8_t* scaled = prep + kt * 8 * (4 * kG);       // V's scales of the part
                weigh(kt, pt);
                // Values' codes: four elements of every group for the four keys, and scales.
                uint32_t vw[2][2][kG / 2], vsc[2][kG];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) lds(at + kSP * K::kCodes + (kt * 16 + 8 * i + ((2 * c + y) ^ c)) * (D / 2) + r * (D / 16), vw[i][y]);
                    lds(scaled + K::kVPairs + ((c ^ (c >> 1)) + 4 * i) * (4 * kG), vsc[i]);
                }
#pragma unroll
                for (int j = 0; j < kG / 2; ++j) {
                    uint32_t x[2][2][4];             // [keys 2c .., keys 2c + 8 ..][codes 0 and 2, 1 and 3][group 2j: two, group 2j + 1: two]
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t u0 = vw[i][0][j], u1 = vw[i][1][j];
                        const uint32_t even = (u0 & 0x0f0f0f0fu) | (u1 << 4 & 0xf0f0f0f0u), odd = (u0 >> 4 & 0x0f0f0f0fu) | (u1 & 0xf0f0f0f0u);
                        codes_f16(even, x[i][0][0], x[i][0][1], x[i][0][2], x[i][0][3]);
                        codes_f16(odd, x[i][1][0], x[i][1][1], x[i][1][2], x[i][1][3]);
                    }
#pragma unroll
                    for (int gg = 0; gg < 2; ++gg) {
                        const int g = 2 * j + gg;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t b0 = hmul2(pt[nt][0], vsc[0][g]), b1 = hmul2(pt[nt][1], vsc[1][g]);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                mma_f16(o[g][h][nt], x[0][0][2 * gg + h], x[0][1][2 * gg + h], x[1][0][2 * gg + h], x[1][1][2 * gg + h], b0, b1);
                        }
                    }
                }
            }
            __syncwarp();
            if (sub == kSteps - 1 || p + kParts >= it.p1) {
                ++read;
                if (++slot == kRing) {
                    slot = 0;
                    phase ^= 1;
                }
                copy();
            }
        }
        if (!ok) break;
        // O's elements 32 g + 4 r to + 3 of rows 2c and 2c + 1.
        const int e0 = 4 * r;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 4);
                l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 8);
                l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 16);
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = nt * 8 + 2 * c + i;
                if (x >= it.rows) continue;
                if (it.whole) {
                    const uint32_t row = (uint32_t)it.rb * K::kRows + x;
                    const int tok = (int)(row / (uint32_t)a.G), h = it.hk * a.G + (int)row - tok * a.G;
                    const float inv = l[nt][i] == 0.f ? 0.f : 1.f / l[nt][i];
                    const long long tt = it.c0 + tok;
                    __nv_bfloat16* dst = a.o + (tt * a.Hq + h) * D + e0;
#pragma unroll
                    for (int g = 0; g < kG; ++g)
                        *reinterpret_cast<uint2*>(dst + 32 * g) = make_uint2(pack_bf16x2(o[g][0][nt][i] * inv, o[g][0][nt][2 + i] * inv),
                                                                             pack_bf16x2(o[g][1][nt][i] * inv, o[g][1][nt][2 + i] * inv));
                    if (r == 0) a.lse[(long long)h * a.T + tt] = l[nt][i] == 0.f ? -INFINITY : (m[nt][i] + __log2f(l[nt][i])) * 0.69314718055994531f;
                } else {
                    const long long row = (long long)it.seg * K::kRows + x;
                    float* dst = a.seg + row * D + e0;
#pragma unroll
                    for (int g = 0; g < kG; ++g)
                        *reinterpret_cast<float4*>(dst + 32 * g) = make_float4(o[g][0][nt][i], o[g][0][nt][2 + i], o[g][1][nt][i], o[g][1][nt][2 + i]);
                    if (r == 0) a.ml[row] = make_float2(m[nt][i], l[nt][i]);
                }
            }
    }
    // Every copy lands before the block ends (after a wait that gave up, too).
    const uint64_t t0 = globaltimer_ns();
    for (; read < issued; ++read) {
        while (!mbar_try_wait(smem_u32(&full[slot]), phase) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        if (++slot == kRing) {
            slot = 0;
            phase ^= 1;
        }
    }
    __syncwarp();
    if (!ok && lane == 0 && atomicCAS(&a.status->code, 0, kStatusTimeout) == 0) {
        a.status->where = 112;
        a.status->block = blockIdx.x;
    }
}

// ----------------------------------------------------------------- more rows

// Items of N rows on the fifth-generation tensor cores: a CTA is a worker, 128 keys a
// tile.  Codes become fp16 and are scaled on the way (by a row's scales relative to its
// largest, times 2^10: with a code exact in fp16), in the order in which a row's codes
// lie; Q has the same order, and O's is undone where it is written.  S^T = K Q^T has keys
// as lanes and K in tensor memory, O^T = V^T P^T elements of d as lanes and V in shared
// memory, read across its rows.  (With K in shared memory too, its tile written and read
// there took as long as V's: 107 us where this took 104.)
//
// What bounds it: a product of 128 x N x 16 takes about 50 (K) and 80 (V) cycles for its
// 128 rows, whatever N up to 32 is: 2050 cycles for 128 keys of 256, 58 % of a CTA's
// time (32 rows over up to 16384 keys); issue slots 61 %; a chain from scores to weights
// of 2700, tiles one after another.  HBM takes 1490.  At d = 128 and 64 the chain is all:
// 2000 cycles a tile.  64 requests of 8192 keys and 8 heads: 16 rows of 256 326 us, 32
// rows 353, 32 rows of 128 243, of 64 219; with m16n8k16 and one, two or four warps an item
// 362 (16 of 256), 352 and 236; 16 rows of 128 this way 226, and 184 by single warps.
// Without gain: row numbers loaded before the wait for the scores (registers), a flag and
// weights worked out before it is looked at instead of a barrier a tile (89 us 94),
// sixteen warps for the softmax and half as many that expand (32 rows of 128 250, of 64
// 210).
template <int D, int N> struct Mid {
    // An item's start and end take as long as 8 to 12 units.  With 4, 8, 12, 16 and 24 (us), 32 rows: 100 requests of up
    // to 16384 keys, one head: of 256 91.0 86.0 86.3 88.5 90.7, of 128 61.7 59.6 60.3 62.5 64.7, of 64 56.2 54.3 55.1 56.5
    // 58.9; 300 requests of up to 1500, two heads: of 256 115 104 101 106 109, of 128 74.0 66.4 65.6 67.7 70.2, of 64 65.2
    // 57.6 58.0 58.7 61.8; 64 requests of 8192: within 3 % of each other up to 12.
    static constexpr int kRows = N, kExtra = 12, kThreads = 896, kWorkers = 1, kHalves = D == 256 ? 2 : 1;
    static constexpr int kRing = D == 256 ? 2 : 4;       // slots of K (codes, both scales) and of V (codes)
    static constexpr uint32_t kCodes = 8 * D, kScales = D / 2, kSlotK = 8 * (kCodes + 2 * kScales), kSlotV = 8 * kCodes;
    static constexpr uint32_t kBox = 128 * 128, kTile = D / 64 * kBox, kQBox = N * 128;      // 64 elements of 128 keys, of N rows
    static constexpr int kWeights = D == 256 ? 1 : 2;    // tiles of weights (of V's rows, two)
    static constexpr uint32_t kP1 = 128 * 2 * N, kV = 0, kQ = 2 * kTile, kP = kQ + D / 64 * kQBox, kRawK = kP + kWeights * kP1, kRawV = kRawK + kRing * kSlotK;
    // What the softmax wants of four tiles' keys; rows of two items: less their maximum, what
    // a sum is multiplied by, keys seen; factors, maxima or sums of four quarters.
    static constexpr uint32_t kKeys = kRawV + kRing * kSlotV, kRows2 = kKeys + 4 * 128 * 4, kRowF = kRows2 + 2 * 3 * N * 4, kRowX = kRowF + N * 4, kWarp = kRowX + 4 * N * 4;
    // Tensor memory: scores of two tiles, O, K's rows of two tiles.
    static constexpr uint32_t kColO = 2 * N, kColK = kColO + kHalves * N, kColumns = kColK + D <= 256 ? 256 : 512;
    static_assert((N == 32 || (N == 16 && D == 256)) && (D == 64 || D == 128 || D == 256) && kExtra <= kExtraMost, "sizes built");
    static_assert(kRawK % 1024 == 0 && kWarp % 16 == 0 && kWarp + table_bytes(kTableMost) + 1024 <= 232448, "shared memory plan");
};
struct MidShared : KvScan {
    uint64_t k_raw_full[4], k_raw_empty[4], v_raw_full[4], v_raw_empty[4], k_full[2], v_full[2], q_full, s_full[2], p_full[2], pv_done[2], drain[2];
    uint32_t live[4], tmem;
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn_major, int b_mn_major) {
    return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// S^T = K Q^T: K in tensor memory (eight columns a step of 16), Q K-major.
template <int D, int N> __device__ __forceinline__ void mid_scores(uint32_t s, uint32_t k_tmem, uint32_t q_smem) {
    using K = Mid<D, N>;
    constexpr uint32_t idesc = idesc_f16_f32(128, N, 0, 0);
    const uint64_t bd = sdesc_sw128(q_smem, 16, 1024);
    static_for<D / 16>([&](auto kc) {
        constexpr uint32_t k = kc, bo = ((k >> 2) * K::kQBox + (k & 3) * 32) >> 4;
        umma_ts_k<8 * k, bo>(s, k_tmem, bd, idesc, k > 0 ? 1u : 0u);
    });
}
// O^T (+)= V^T P^T for 128 (64) of d, both MN-major: V's rows (boxes of 64 elements), P's
// rows of N weights a key, 2 N bytes apart and swizzled over as many.
template <int D, int N> __device__ __forceinline__ void mid_values(uint32_t o, uint32_t v_smem, uint32_t p_smem, uint32_t acc) {
    using K = Mid<D, N>;
    constexpr uint32_t idesc = idesc_f16_f32(D == 64 ? 64 : 128, N, 1, 1);
    constexpr uint64_t kOther = (uint64_t)(N == 32 ? 4 ^ 2 : 6 ^ 2) << 61;      // 64- or 32-byte swizzle for 128
    const uint64_t ad = sdesc_sw128(v_smem, K::kBox, 1024), bd = sdesc_sw128(p_smem, 16, 16 * N) ^ kOther;
    static_for<8>([&](auto kc) {
        constexpr uint32_t k = kc, ao = (k * 2048) >> 4, bo = (k * 32 * N) >> 4;
        umma_ss_k<ao, bo>(o, ad, bd, idesc, (acc | k) != 0);
    });
}

// A key's scales (f16 pairs) times 2^(26 - field), each twice; returns the exponent
// field of the largest (1 to 30), or 0 where all are 0.
template <int D> __device__ __forceinline__ uint32_t mid_scales(const uint32_t (&h)[D / 64], uint32_t (&sc)[D / 32]) {
    uint32_t m = h[0];
#pragma unroll
    for (int i = 1; i < D / 64; ++i) m = hmax2(m, h[i]);
    m = hmax2(m, __byte_perm(m, m, 0x1032));
    const uint32_t ex = hmin2(hmax2(m, 0x04000400u), 0x78007800u) & 0x7c007c00u;
    // 2^(26 - field) in one step where it is below 2^16, else after 2^(16 - field): exact
    // (the products are multiples of 2^-21).
    const bool one = ex >= 0x2c002c00u;
    const uint32_t f = (one ? 0xa400a400u : 0x7c007c00u) - ex, f2 = one ? 0x3c003c00u : 0x64006400u;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint32_t x = hmul2(hmul2(h[i], f), f2);
        sc[2 * i] = __byte_perm(x, x, 0x1010);
        sc[2 * i + 1] = __byte_perm(x, x, 0x3232);
    }
    return m ? ex >> 26 : 0;
}
// Half of a key's codes into its row of a tile.  Lanes are keys; which 16 bytes each
// takes first depends on its key, so that neither loads nor stores meet in a bank.
template <int D> __device__ __forceinline__ void mid_expand(const uint8_t* codes, uint8_t* tile, int key, int half, const uint32_t (&sc)[D / 32]) {
    constexpr int kC = D / 32, kG = D / 32;      // 16-byte pieces of a row
    const int turn = (D == 256 ? key : D == 128 ? key >> 1 : 0) + half * (kC / 2);
    const uint8_t* row = codes + key * (D / 2);
    uint8_t* to = tile + key * 128;
    uint32_t w[kC / 2][4];
#pragma unroll
    for (int j = 0; j < kC / 2; ++j) lds(row + ((j + turn) & (kC - 1)) * 16, w[j]);
#pragma unroll
    for (int j = 0; j < kC / 2; ++j) {
        const int c = (j + turn) & (kC - 1);
        uint8_t* box = to + (c >> 1) * (128 * 128);
        const int first = (c & 1) * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t x[4];
            codes_f16(w[j][k], x[0], x[1], x[2], x[3]);
            constexpr int kMask = kG - 1;
            x[0] = hmul2(x[0], sc[2 * k & kMask]);
            x[1] = hmul2(x[1], sc[2 * k & kMask]);
            x[2] = hmul2(x[2], sc[(2 * k & kMask) + 1]);
            x[3] = hmul2(x[3], sc[(2 * k & kMask) + 1]);
            sts(box + (((first + k) ^ (key & 7)) * 16), x);
        }
    }
}
// Half of a key's codes into its lane of tensor memory.  A row's pieces are loaded in an
// order that depends on the lane (two lanes of eight meet in a bank instead of eight)
// and put back in order by selections.
template <int D> __device__ __forceinline__ void mid_expand_lane(const uint8_t* codes, uint32_t to, int key, int half, const uint32_t (&sc)[D / 32]) {
    constexpr int kC = D / 64, kG = D / 32;      // 16-byte pieces of half a row
    const int turn = D == 256 ? key : key >> 1;
    const uint8_t* row = codes + key * (D / 2) + half * (D / 4);
    uint32_t w[kC][4];
#pragma unroll
    for (int j = 0; j < kC; ++j) lds(row + ((j + turn) & (kC - 1)) * 16, w[j]);
#pragma unroll
    for (int o = 1; o < kC; o *= 2) {            // piece c is where (c - turn) was
        uint32_t y[kC][4];
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[c][k] = turn & o ? w[(c - o) & (kC - 1)][k] : w[c][k];
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) w[c][k] = y[c][k];
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        uint32_t x[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            constexpr int kMask = kG - 1;
            codes_f16(w[c][k], x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
            x[4 * k] = hmul2(x[4 * k], sc[2 * k & kMask]);
            x[4 * k + 1] = hmul2(x[4 * k + 1], sc[2 * k & kMask]);
            x[4 * k + 2] = hmul2(x[4 * k + 2], sc[(2 * k & kMask) + 1]);
            x[4 * k + 3] = hmul2(x[4 * k + 3], sc[(2 * k & kMask) + 1]);
        }
        tmem_st16(to + half * (D / 4) + c * 16, x);
    }
    tmem_wait_st();
}
// The element that position x of a row's codes is.
template <int D> __device__ __forceinline__ int element_at(int x) {
    const int u = x >> 2;
    return u % (D / 32) * 32 + u / (D / 32) * 4 + (x & 3);
}
// For each of N columns, op over the warp's lanes: lane l gets column l % N.
template <int N, class Op> __device__ __forceinline__ float over_lanes(float (&v)[N], int lane, const Op& op) {
#pragma unroll
    for (int o = N / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = lane & o ? v[i + o] : v[i], send = lane & o ? v[i] : v[i + o];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
#pragma unroll
    for (int o = N; o < 32; o *= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    return v[0];
}
template <int N> __device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[N]) {
    if constexpr (N == 16) tmem_ld16(at, r);
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(at));
    tmem_wait_ld();
}
template <int N> __device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[N]) {
    if constexpr (N == 16) tmem_st16(at, r);
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A barrier of the softmax's 256 threads, and one with the `or` of a flag over them.
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_or(bool x) {
    uint32_t y;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y) : "r"((uint32_t)x) : "memory");
    return y != 0;
}

// Warps 0 to 7 do the softmax (a quarter of the keys, at the end of d, and half the rows
// each), 8 to 15 expand K and 16 to 23 V (two threads a key), 24 and 25 copy, 26 and 27
// issue the two products.
template <int D, int N>
__global__ void __launch_bounds__(896, 1) kv4_mid_kernel(const KvArgs a) {
    using K = Mid<D, N>;
    using Walk = KvWalk<N, K::kExtra>;
    constexpr int kG = D / 32, kC = N / 2;
    constexpr uint32_t kRing = K::kRing;
    extern __shared__ __align__(1024) uint8_t dsmem_tiles[];
    __shared__ MidShared sh;
    uint8_t* const dsmem = dsmem_tiles;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    KvTables t;
    t.pref = a.B <= kTableMost ? reinterpret_cast<int*>(dsmem + K::kWarp) : a.tables + (long long)blockIdx.x * (4 * a.B + 3);
    t.items = t.pref + a.B + 1;
    t.cu = t.items + a.B + 1;
    t.len = t.cu + a.B + 1;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.k_raw_full[i], 1);
            mbar_init(&sh.k_raw_empty[i], 16);
            mbar_init(&sh.v_raw_full[i], 1);
            mbar_init(&sh.v_raw_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.k_full[i], 8);
            mbar_init(&sh.v_full[i], 8);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 8);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.drain[i], 1);
        }
        mbar_init(&sh.q_full, 8);
        fence_mbar_init();
        sh.abort_flag = 0;
    }
    if (warp == 26) {
        tmem_alloc(&sh.tmem, K::kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    grid_launch_next();
    grid_wait();
    prefetch_tables<K>(a, tid);
    const KvHeader hdr = build_tables<K>(a, t, sh, tid);
    fill_rows<K>(a, t, tid);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem, smem = smem_u32(dsmem);
    // Exponent field of K's largest scale, V's e, the tile's parts that are there.
    uint32_t* const keys = reinterpret_cast<uint32_t*>(dsmem + K::kKeys);
    Walk walk;
    walk.start(a, t, hdr, blockIdx.x);
    KvItem it;
    bool ok = true;
    uint32_t tile = 0;                               // tiles of this CTA so far
    // What is done once a tile is told by two barriers in turn.
    auto wait2 = [&](uint64_t (&bars)[2], uint32_t x) -> bool { return kv_wait(&bars[x & 1], x >> 1 & 1, &sh.abort_flag); };
    // 896 threads of 72 registers: 2 x 104, 4 x 64 and 40 by 128 threads are as many.
    if (warp < 8) {
        regs_inc<104>();
        const int quarter = warp & 3, c0 = (warp >> 2) * kC, key = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)quarter << 21) + c0;
        float *const row_f = reinterpret_cast<float*>(dsmem + K::kRowF) + c0, *const row_x = reinterpret_cast<float*>(dsmem + K::kRowX) + c0;
        // Its weights: 16-byte pieces, swizzled.
        uint8_t* const p_key = dsmem + K::kP + key * (2 * N);
        const int p_piece = N == 32 ? c0 / 8 ^ (key >> 1 & 3) : c0 / 8 ^ (key >> 2 & 1);
        // An item's Q in the codes' order, scaled by a power of two, and its rows' numbers.
        auto stage = [&](const KvItem& item, uint32_t which) {
            float* const rows = reinterpret_cast<float*>(dsmem + K::kRows2) + which * (3 * N);
            constexpr int kW = D / 8, kPer = 32 / kW, kPasses = N / 8 / kPer;      // 16-byte pieces of a row of fp16; rows a pass
            const int w = lane % kW, e0 = element_at<D>(8 * w);
            uint2 in[kPasses][2];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int x = (warp * kPasses + i) * kPer + lane / kW;
                const uint32_t row = (uint32_t)item.rb * N + x;
                const int tok = (int)(row / (uint32_t)a.G), h = (int)row - tok * a.G;
                in[i][0] = in[i][1] = make_uint2(0, 0);
                if (x < item.rows) {
                    const __nv_bfloat16* src = a.q + (long long)(item.c0 + tok) * a.q_stride + (item.hk * a.G + h) * D + e0;
                    in[i][0] = *reinterpret_cast<const uint2*>(src);
                    in[i][1] = *reinterpret_cast<const uint2*>(src + 32);
                }
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int x = (warp * kPasses + i) * kPer + lane / kW;
                const uint32_t v[4] = {in[i][0].x, in[i][0].y, in[i][1].x, in[i][1].y};
                float most = 0.f;
#pragma unroll
                for (int y = 0; y < 4; ++y) most = fmax3(most, fabsf(__uint_as_float(v[y] << 16)), fabsf(__uint_as_float(v[y] & 0xffff0000u)));
#pragma unroll
                for (int o = kW / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                const int e = min(max((int)(__float_as_uint(most) >> 23), kQLift + 1), 254);
                const float down = __uint_as_float((uint32_t)(254 + kQLift - e) << 23);
                uint32_t q[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) q[y] = pack_f16x2(__uint_as_float(v[y] << 16) * down, __uint_as_float(v[y] & 0xffff0000u) * down);
                sts(dsmem + K::kQ + (w >> 3) * K::kQBox + x * 128 + ((w & 7) ^ (x & 7)) * 16, q);
                if (w == 0) {
                    rows[N + x] = a.scale_log2 * __uint_as_float((uint32_t)(e - kQLift) << 23);
                    rows[x] = -kNone;
                    reinterpret_cast<int*>(rows)[2 * N + x] = min(item.s, item.s - item.n + (int)(((uint32_t)item.rb * N + x) / (uint32_t)a.G) + 1);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full);
        };
        KvItem coming;
        bool more = walk.next(a, t, coming);
        if (more) stage(coming, 0);
        for (uint32_t which = 0; ok && more; which ^= 1) {
            it = coming;
            soft_sync();                             // its rows' numbers are there, those of the one before read
            float *const row_m = reinterpret_cast<float*>(dsmem + K::kRows2) + which * (3 * N) + c0, *const row_up = row_m + N;
            int* const row_lim = reinterpret_cast<int*>(row_up + N);
            const int lim_min = row_lim[0];
            uint64_t l[kC / 2];
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) l[i] = 0;
            for (int p = it.p0; p < it.p1; p += 8, ++tile) {
                ok = wait2(sh.s_full, tile) && ok;
                tc_fence_after();
                uint32_t r[kC];
                tmem_ld<kC>(lanes + (tile & 1) * N, r);
                // K's scale is 2^(field - 26) times what it was expanded with.
                const uint32_t info = keys[(tile & 3) * 128 + key], here = info >> 16;
                const float ek = __uint_as_float((101u + (info & 255u)) << 23), ev = value_e(info >> 8 & 255u), back = value_back(info >> 8 & 255u);
                float z[kC], most = -INFINITY;
#pragma unroll
                for (int i = 0; i < kC; i += 2)
                    f2_unpack(f2_fma(f2_mul(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f2_pack(ek, ek)), *reinterpret_cast<const uint64_t*>(row_up + i), f2_pack(ev, ev)), z[i], z[i + 1]);
                if (p * 16 + 128 > lim_min || here != 255u) {
                    const bool gone = !(here >> (key >> 4) & 1u);
#pragma unroll
                    for (int i = 0; i < kC; ++i)
                        if (gone || p * 16 + key >= row_lim[i]) z[i] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < kC; i += 2) {
                    float y[2];
                    f2_unpack(f2_add(f2_pack(z[i], z[i + 1]), *reinterpret_cast<const uint64_t*>(row_m + i)), y[0], y[1]);
                    most = fmax3(most, y[0], y[1]);
                }
                // O and l follow a row's running maximum as above.
                if (soft_or(most > kTau + kLift || !ok)) {
                    if (ok && tile) ok = wait2(sh.pv_done, tile - 1);
                    ok = !soft_or(!ok);
                    if (!ok) break;
                    tc_fence_after();
                    float v[kC];
#pragma unroll
                    for (int i = 0; i < kC; ++i) v[i] = z[i];
                    const float x = over_lanes<kC>(v, lane, [](float y, float u) { return fmaxf(y, u); });
                    if (lane < kC) row_x[quarter * N + lane] = x;
                    soft_sync();
                    if (quarter == 0 && lane < kC) {
                        const float m = -row_m[lane], next = fmaxf(m, fmaxf(fmaxf(row_x[lane], row_x[N + lane]), fmaxf(row_x[2 * N + lane], row_x[3 * N + lane])) - kLift);
                        row_f[lane] = ex2_mufu(m - next);
                        row_m[lane] = -next;
                    }
                    soft_sync();
#pragma unroll
                    for (int i = 0; i < kC; i += 2) l[i / 2] = f2_mul(l[i / 2], *reinterpret_cast<const uint64_t*>(row_f + i));
                    if (p > it.p0) {
#pragma unroll
                        for (int h = 0; h < K::kHalves; ++h) {
                            tmem_ld<kC>(lanes + K::kColO + N * h, r);
#pragma unroll
                            for (int i = 0; i < kC; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * row_f[i]);
                            tmem_st<kC>(lanes + K::kColO + N * h, r);
                        }
                        tmem_wait_st();
                    }
                }
                uint32_t weights[kC / 2];
#pragma unroll
                for (int i = 0; i < kC; i += 2) {
                    float y[2];
                    f2_unpack(f2_add(f2_pack(z[i], z[i + 1]), *reinterpret_cast<const uint64_t*>(row_m + i)), y[0], y[1]);
                    y[0] = ex2_mufu(y[0]);
                    y[1] = ex2_mufu(y[1]);
                    l[i / 2] = f2_fma(f2_pack(y[0], y[1]), f2_pack(back, back), l[i / 2]);
                    weights[i / 2] = pack_f16x2(y[0], y[1]);
                }
                // The weights that were here are multiplied (with two tiles of them, before these
                // scores were).
                if (K::kWeights == 1 && tile) ok = wait2(sh.pv_done, tile - 1) && ok;
                uint8_t* const to = p_key + (K::kWeights == 2 && (tile & 1) ? K::kP1 : 0);
#pragma unroll
                for (int i = 0; i < kC / 8; ++i)
                    *reinterpret_cast<uint4*>(to + ((p_piece ^ i) << 4)) = make_uint4(weights[4 * i], weights[4 * i + 1], weights[4 * i + 2], weights[4 * i + 3]);
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[tile & 1]);
            }
            // The next item's Q, whose first scores are then there when this one is written.
            if (ok) {
                more = walk.next(a, t, coming);
                if (more) stage(coming, which ^ 1);
                ok = wait2(sh.pv_done, tile - 1);
            }
            tc_fence_after();
            float v[kC];
#pragma unroll
            for (int i = 0; i < kC; i += 2) f2_unpack(l[i / 2], v[i], v[i + 1]);
            const float sum = over_lanes<kC>(v, lane, [](float x, float y) { return x + y; });
            if (lane < kC) row_x[quarter * N + lane] = sum;
            ok = !soft_or(!ok);
            if (!ok) break;
            if (quarter == 0 && lane < kC) {
                const float total = row_x[lane] + row_x[N + lane] + row_x[2 * N + lane] + row_x[3 * N + lane], m = -row_m[lane];
                // V's rows are 2^10 times what they stand for.
                row_f[lane] = !it.whole ? 0.0009765625f : total == 0.f ? 0.f : 0.0009765625f / total;
                if (c0 + lane < it.rows) {
                    if (it.whole) {
                        const uint32_t row = (uint32_t)it.rb * N + c0 + lane;
                        const int tok = (int)(row / (uint32_t)a.G), h = it.hk * a.G + (int)row - tok * a.G;
                        a.lse[(long long)h * a.T + it.c0 + tok] = total == 0.f ? -INFINITY : (m + __log2f(total)) * 0.69314718055994531f;
                    } else {
                        a.ml[(long long)it.seg * N + c0 + lane] = make_float2(m, total);
                    }
                }
            }
            soft_sync();
#pragma unroll
            for (int h = 0; h < K::kHalves; ++h) {
                uint32_t r[kC];
                tmem_ld<kC>(lanes + K::kColO + N * h, r);
                // Four lanes hold four neighbours of every row: each takes one row of four.  (64
                // elements are in the first 16 lanes of each quarter.)
                const int e = element_at<D>((D == 64 ? quarter * 16 + (lane & 15) : h * 128 + key) & ~3), q = lane & 3;
#pragma unroll
                for (int i = 0; i < kC; i += 4) {
#pragma unroll
                    for (int j = i; j < i + 4; j += 2) {
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, q & 1 ? r[j] : r[j + 1], 1);
                        if (q & 1) r[j] = other; else r[j + 1] = other;
                    }
#pragma unroll
                    for (int j = i; j < i + 2; ++j) {
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, q & 2 ? r[j] : r[j + 2], 2);
                        if (q & 2) r[j] = other; else r[j + 2] = other;
                    }
                }
#pragma unroll
                for (int i = 0; i < kC; i += 4) {
                    const int x = c0 + i + q;
                    if (x >= it.rows || (D == 64 && lane >= 16)) break;
                    const float f = row_f[i + q];
                    float y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = f == 0.f ? 0.f : __uint_as_float(r[i + j]) * f;
                    if (it.whole) {
                        const uint32_t row = (uint32_t)it.rb * N + x;
                        const int tok = (int)(row / (uint32_t)a.G), hh = (int)row - tok * a.G;
                        *reinterpret_cast<uint2*>(a.o + ((long long)(it.c0 + tok) * a.Hq + it.hk * a.G + hh) * D + e) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                    } else {
                        *reinterpret_cast<float4*>(a.seg + ((long long)it.seg * N + x) * D + e) = make_float4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
        }
    } else if (warp < 24) {
        regs_dec<64>();
      if (warp < 16) {
        const int key = tid & 127, half = warp >= 12;
        while (ok && walk.next(a, t, it)) {
            for (int p = it.p0; p < it.p1; p += 8, ++tile) {
                const uint32_t slot = tile % kRing;
                const uint8_t *const raw = dsmem + K::kRawK + slot * K::kSlotK, *const ks = raw + 8 * K::kCodes, *const vs = ks + 8 * K::kScales;
                if (!(ok = kv_wait(&sh.k_raw_full[slot], tile / kRing & 1, &sh.abort_flag))) break;
                const uint32_t here = sh.live[slot];
                const bool real = (here >> (key >> 4) & 1u) && p * 16 + key < it.seen;
                uint32_t h[D / 64], sc[kG];
                scale_pairs<D>(vs + key * kG, real, h);
                const uint32_t fv = mid_scales<D>(h, sc);
                scale_pairs<D>(ks + key * kG, true, h);
                const uint32_t fk = mid_scales<D>(h, sc);
                // The tile before the last is done with its rows.
                if (tile >= 2 && !(ok = wait2(sh.s_full, tile - 2))) break;
                tc_fence_after();
                if (!half) keys[(tile & 3) * 128 + key] = fk | (fv ? fv + kValue : kNoValue) << 8 | here << 16;
                mid_expand_lane<D>(raw, tmem + ((uint32_t)(warp & 3) << 21) + K::kColK + (tile & 1) * (D / 2), key, half, sc);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.k_full[tile & 1]);
                    mbar_arrive(&sh.k_raw_empty[slot]);
                }
            }
        }
      } else {
        const int key = tid & 127, half = warp >= 20;
        bool more = walk.next(a, t, it);
        int p = it.p0;
        // V's scales come with K: those of the next tile are taken first, so that its copies
        // need not wait for this one's V.
        auto take = [&](uint32_t (&h)[D / 64]) -> bool {
            const uint32_t slot = tile % kRing;
            if (!kv_wait(&sh.k_raw_full[slot], tile / kRing & 1, &sh.abort_flag)) return false;
            const bool real = (sh.live[slot] >> (key >> 4) & 1u) && p * 16 + key < it.seen;
            scale_pairs<D>(dsmem + K::kRawK + slot * K::kSlotK + 8 * (K::kCodes + K::kScales) + key * kG, real, h);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.k_raw_empty[slot]);
            ++tile;
            p += 8;
            if (p >= it.p1) {
                more = walk.next(a, t, it);
                p = it.p0;
            }
            return true;
        };
        uint32_t now[D / 64], next[D / 64] = {};
        if (more) ok = take(now);
        for (uint32_t done = 0; ok && done < tile; ++done) {
            if (more && !(ok = take(next))) break;
            const uint32_t slot = done % kRing;
            uint32_t sc[kG];
            mid_scales<D>(now, sc);
            if (!(ok = kv_wait(&sh.v_raw_full[slot], done / kRing & 1, &sh.abort_flag))) break;
            if (done >= 2 && !(ok = wait2(sh.pv_done, done - 2))) break;
            mid_expand<D>(dsmem + K::kRawV + slot * K::kSlotV, dsmem + K::kV + (done & 1) * K::kTile, key, half, sc);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.v_full[done & 1]);
                mbar_arrive(&sh.v_raw_empty[slot]);
            }
#pragma unroll
            for (int i = 0; i < D / 64; ++i) now[i] = next[i];
        }
      }
    } else {
        regs_dec<40>();
      if (warp < 26) {
        // K's codes and both scales, or V's codes: one copy for the parts of a tile that
        // are in one page (a copy costs its warp 85 cycles).
        const bool v = warp == 25;
        uint64_t *const full = v ? sh.v_raw_full : sh.k_raw_full, *const empty = v ? sh.v_raw_empty : sh.k_raw_empty;
        const int what = lane & 3, which = lane >> 2, run_log2 = a.ps_log2 - 4;
        const bool copies = v ? what == 0 : what < 3;
        const uint8_t* const from = v ? a.vp : what == 0 ? a.kp : what == 1 ? a.ks : a.vs;
        const uint32_t bytes = what == 0 ? K::kCodes : K::kScales, slot_bytes = v ? K::kSlotV : K::kSlotK, part_bytes = slot_bytes / 8;
        const uint32_t into = smem + (v ? K::kRawV : K::kRawK) + (what == 0 ? 0 : 8 * K::kCodes + (what - 1) * 8 * K::kScales) + which * bytes;
        while (ok && walk.next(a, t, it)) {
            auto pages = [&](int p) -> int {         // of parts p .. p + 31
                if (p + lane >= it.p1) return -1;
                const int x = a.table[(long long)it.b * a.W + ((p + lane) * 16 >> a.ps_log2)];
                return x >= 0 && x < a.P ? x : -1;
            };
            int win = pages(it.p0), win_next = pages(it.p0 + 32);
            for (int p = it.p0; p < it.p1; p += 8, ++tile) {
                if (p != it.p0 && ((p - it.p0) & 31) == 0) {
                    win = win_next;
                    win_next = pages(p + 32);
                }
                const uint32_t slot = tile % kRing;
                if (tile >= kRing && !(ok = kv_wait(&empty[slot], (tile / kRing & 1) ^ 1, &sh.abort_flag))) break;
                const int page = __shfl_sync(0xffffffffu, win, (p - it.p0 + which) & 31);
                const uint32_t on4 = __ballot_sync(0xffffffffu, what == 0 && page >= 0);      // bit 4 i: part i
                if (lane == 0) {
                    if (!v) {
                        uint32_t on = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) on |= (on4 >> (4 * i) & 1u) << i;
                        sh.live[slot] = on;
                    }
                    if (on4) mbar_arrive_expect_tx(&full[slot], part_bytes * __popc(on4));
                    else mbar_arrive(&full[slot]);
                }
                __syncwarp();
                const int in_page = (p + which) & ((1 << run_log2) - 1);
                if (copies && page >= 0 && (which == 0 || in_page == 0)) {
                    const int run = min(min((1 << run_log2) - in_page, 8 - which), it.p1 - p - which);
                    const long long row = (((long long)page * a.Hkv + it.hk) << a.ps_log2) + in_page * 16;
                    bulk_load(into + slot * slot_bytes, from + row * (what == 0 ? D / 2 : D / 32), run * bytes, &full[slot]);
                }
            }
        }
        // Every copy lands before the block ends.
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = tile < kRing ? 0 : tile - kRing; i < tile; ++i)
            while (!mbar_try_wait(smem_u32(&full[i % kRing]), i / kRing & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {}
      } else {
        // Scores, and weighted values, by a warp each: one that waits holds up its own only.
        const bool values = warp == 27;
        uint32_t items = 0;
        while (ok && walk.next(a, t, it)) {
            if (!values && !(ok = kv_wait(&sh.q_full, items++ & 1, &sh.abort_flag))) break;
            for (int p = it.p0; p < it.p1; p += 8, ++tile) {
                if (values) {
                    if (!(ok = wait2(sh.v_full, tile) && wait2(sh.p_full, tile))) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < K::kHalves; ++h)
                        mid_values<D, N>(tmem + K::kColO + N * h, smem + K::kV + (tile & 1) * K::kTile + h * 2 * K::kBox, smem + K::kP + (K::kWeights == 2 && (tile & 1) ? K::kP1 : 0), p > it.p0);
                    umma_commit_w(&sh.pv_done[tile & 1]);
                } else {
                    // The scores that were here are read and their weights multiplied.
                    if (!(ok = wait2(sh.k_full, tile) && (tile < 2 || wait2(sh.pv_done, tile - 2)))) break;
                    tc_fence_after();
                    mid_scores<D, N>(tmem + (tile & 1) * N, tmem + K::kColK + (tile & 1) * (D / 2), smem + K::kQ);
                    umma_commit_w(&sh.s_full[tile & 1]);
                }
            }
        }
        if (!ok) {                                   // products in flight end before their memory is given back
            umma_commit_w(&sh.drain[values]);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&sh.drain[values]), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
      }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sh.abort_flag && atomicCAS(&a.status->code, 0, kStatusTimeout) == 0) {
        a.status->where = 113;
        a.status->block = blockIdx.x;
    }
    if (warp == 26) tmem_dealloc(tmem, K::kColumns);
}

// Joins the segments of a row (of one head) that a range's end has cut; writes the
// rows without a key.  A warp a row, or with few rows a block of eight.
template <int D, bool kSplit, int kExtra>
__global__ void __launch_bounds__(256) kv4_join_kernel(const KvArgs a, int rows_item) {
    constexpr int E = D / 32;
    __shared__ float s_o[kSplit ? 8 : 1][kSplit ? D : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long w = kSplit ? blockIdx.x : blockIdx.x * 8LL + warp;
    if (w >= (long long)a.T * a.Hq) return;
    const int t = (int)(w / a.Hq), h = (int)(w - (long long)t * a.Hq), hk = h / a.G;
    grid_wait();
    const KvHeader hdr = *a.hdr;
    const KvRow q = a.rows[t];
    if (hdr.bad || q.n == 0) return;
    const int row = (t - q.c0) * a.G + h - hk * a.G, rb = row / rows_item, in = row - rb * rows_item, nb = row_blocks(q.n, a.G, rows_item);
    const int units = item_units(q.s, kExtra), item = hk * nb + rb, u0 = q.pref + item * units, seen = keys_seen(q.n, q.s, a.G, rb, rows_item);
    const bool some = units > 0 && seen > 0;
    const int first = some ? worker_of(hdr, u0) : 0, all = some ? worker_of(hdr, u0 + units - 1) - first + 1 : 0;
    // Row in the k-th worker's segment, -1: it has none.
    auto place = [&](int k) -> long long {
        if (k >= all) return -1;
        const int from = max(0, unit_of(hdr, first + k) - u0), to = min(units, unit_of(hdr, first + k + 1) - u0);
        int p0, p1;
        parts_of(from, to, seen, kExtra, p0, p1);
        if (p0 >= p1) return -1;
        return p0 == 0 && p1 == (seen + 15) >> 4 ? -2 : (long long)(q.items + item + first + k) * rows_item + in;
    };
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float2 ml;
    long long at;
    auto load = [&](int k) {
        at = place(k);
        ml = at >= 0 ? a.ml[at] : make_float2(-INFINITY, 0.f);
    };
    for (int k0 = all > 0 ? (all - 1) / 32 * 32 : 0; k0 >= 0; k0 -= 32) {
        load(k0 + lane);
        if (__any_sync(0xffffffffu, at == -2)) return;       // written by its one worker
        M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int k0 = 0; k0 < all; k0 += 32) {
        if (k0) load(k0 + lane);
        const float f = ml.y == 0.f ? 0.f : ex2_mufu(ml.x - M);   // a sum of 0: no key seen; a NaN stays one
        L += f * ml.y;
        const int cnt = min(32, all - k0);
#pragma unroll 4
        for (int k = kSplit ? warp : 0; k < cnt; k += kSplit ? 8 : 1) {
            const long long from = __shfl_sync(0xffffffffu, at, k);
            const float fk = __shfl_sync(0xffffffffu, f, k);
            if (from < 0 || fk == 0.f) continue;
            const float* src = a.seg + from * D + lane * E;
            float v[E];
            if constexpr (E == 2) {
                const float2 x = *reinterpret_cast<const float2*>(src);
                v[0] = x.x, v[1] = x.y;
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(src + e);
                    v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(fk, v[e], acc[e]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if constexpr (kSplit) {
#pragma unroll
        for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int e = 0; e < E; ++e)
            for (int y = 1; y < 8; ++y) acc[e] += s_o[y][lane * E + e];
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t out[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + ((long long)t * a.Hq + h) * D) + lane * (E / 2);
    if constexpr (E == 2) *dst = out[0];
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    if (lane == 0) a.lse[(long long)h * a.T + t] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

// -------------------------------------------------------------------- expand

struct ExpandArgs {
    const uint8_t *kp, *ks, *vp, *vs;
    __nv_bfloat16 *ko, *vo;
    const int* list;         // [n] pages, null: page i
    const int* lens;         // [n / W] (null: all): entries past a request's keys are passed over
    int* table;              // [n] or null: takes i where page i was written, else -1
    int n, W, Hkv, P, ps_log2;
};

// A warp takes 16 rows of one page, head and of K or V: four at a time, eight lanes
// a row, whose four loads are made before the first is used.
template <int D>
__global__ void __launch_bounds__(256) kv4_expand_kernel(const ExpandArgs a) {
    constexpr int kG = D / 32;
    grid_launch_next();
    grid_wait();
    const int lane = threadIdx.x & 31, l = lane & 7, ps = 1 << a.ps_log2;
    const long long all = ((long long)a.n * a.Hkv) << (a.ps_log2 - 3);
    for (long long w = blockIdx.x * 8LL + (threadIdx.x >> 5); w < all; w += gridDim.x * 8LL) {
        const bool v = w & 1;
        const int quarter = (int)(w >> 1) & ((ps >> 4) - 1);
        const long long x = w >> (a.ps_log2 - 3);
        const int i = (int)(x / a.Hkv), h = (int)(x - (long long)i * a.Hkv);
        const bool skip = a.lens && ((long long)(i % a.W) << a.ps_log2) >= a.lens[i / a.W];
        const int page = skip ? -1 : a.list ? a.list[i] : i;
        const bool real = page >= 0 && page < a.P;
        if (a.table && !v && h == 0 && quarter == 0 && lane == 0) a.table[i] = real ? i : -1;
        if (!real) continue;
        const long long from = (((long long)page * a.Hkv + h) << a.ps_log2) + quarter * 16 + (lane >> 3);
        const long long to = (((long long)i * a.Hkv + h) << a.ps_log2) + quarter * 16 + (lane >> 3);
        const uint8_t *codes = (v ? a.vp : a.kp) + from * (D / 2) + l * (D / 16), *scales = (v ? a.vs : a.ks) + from * kG;
        __nv_bfloat16* out = (v ? a.vo : a.ko) + to * D + 4 * l;
        uint32_t c[4][kG / 2], s[4][D == 256 ? 2 : 1];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const uint8_t *pc = codes + y * 4 * (D / 2), *pss = scales + y * 4 * kG;
            if constexpr (D == 64) {
                c[y][0] = *reinterpret_cast<const uint32_t*>(pc);
                s[y][0] = *reinterpret_cast<const uint16_t*>(pss);
            } else if constexpr (D == 128) {
                const uint2 u = *reinterpret_cast<const uint2*>(pc);
                c[y][0] = u.x, c[y][1] = u.y;
                s[y][0] = *reinterpret_cast<const uint32_t*>(pss);
            } else {
                const uint4 u = *reinterpret_cast<const uint4*>(pc);
                c[y][0] = u.x, c[y][1] = u.y, c[y][2] = u.z, c[y][3] = u.w;
                const uint2 z = *reinterpret_cast<const uint2*>(pss);
                s[y][0] = z.x, s[y][1] = z.y;
            }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int j = 0; j < kG / 2; ++j) {
                uint32_t p[4];
                codes_f16(c[y][j], p[0], p[1], p[2], p[3]);
#pragma unroll
                for (int gg = 0; gg < 2; ++gg) {
                    const int g = 2 * j + gg;
                    const float sc = scale_f32(s[y][g / 4] >> (g % 4 * 8) & 0xffu);
                    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&p[2 * gg])), hi = __half22float2(*reinterpret_cast<const __half2*>(&p[2 * gg + 1]));
                    *reinterpret_cast<uint2*>(out + (long long)y * 4 * D + 32 * g) = make_uint2(pack_bf16x2(lo.x * sc, lo.y * sc), pack_bf16x2(hi.x * sc, hi.y * sc));
                }
            }
    }
}

// ---------------------------------------------------------------------- host

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

int launch_expand(const ExpandArgs& a, int d, int sms, cudaStream_t stream) {
    const long long all = ((long long)a.n * a.Hkv) << (a.ps_log2 - 3), most = 8LL * sms;
    const long long blocks = (all + 7) / 8;
    auto kern = d == 64 ? kv4_expand_kernel<64> : d == 128 ? kv4_expand_kernel<128> : kv4_expand_kernel<256>;
    return launch_dependent(kern, (int)(blocks < most ? blocks : most), 256, 0, stream, a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// Rows of an item of few rows: eight a product's N.
int item_rows(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

// Workspace of few rows: header, what the rows are, the segments' (m, l) and O.  The
// largest of the three item sizes, so that a workspace for long drafts serves
// single tokens.
struct KvLayout {
    size_t tables, rows, ml, seg, total;
};
KvLayout kv_layout(int T, int B, int Hkv, int G, int d, int sms) {
    size_t most = 0;
    for (int rows = 8; rows <= 32; rows *= 2) {
        const size_t items = (size_t)Hkv * ((long long)T * G / rows + (T < B ? T : B)), workers = (size_t)sms * 16;
        const size_t n = (items + workers) * rows;
        most = n > most ? n : most;
    }
    KvLayout w;
    w.tables = 256;
    w.rows = align256(w.tables + (B > kTableMost ? (size_t)sms * table_bytes(B) : 0));
    w.ml = align256(w.rows + (size_t)T * sizeof(KvRow));
    w.seg = align256(w.ml + most * 8);
    w.total = align256(w.seg + most * d * 4);
    return w;
}

// Workspace of many rows: the expanded pages, the table that names them, and
// fa_prefix_fwd's; 0: this call's pages are too many.
struct ManyLayout {
    size_t k, v, table, prefix, total;
};
ManyLayout many_layout(int T, int B, int Hq, int Hkv, int d, int max_seqlen, int W, int page) {
    ManyLayout w = {};
    const size_t one = (size_t)B * W * page * Hkv * d * 2;
    if (max_seqlen * (long long)(Hq / Hkv) <= many_rows(d) || one > kExpandMost / 2) return w;
    w.v = align256(one);
    w.table = w.v + align256(one);
    w.prefix = align256(w.table + 4 * (size_t)B * W);
    w.total = w.prefix + fa_prefix_workspace_size(T, B, Hq, Hkv, d, max_seqlen);
    return w;
}

template <class K, int D>
int launch_few(void (*kern)(KvArgs), std::atomic<uint64_t>& prepared, const KvArgs& a, int sms, cudaStream_t stream) {
    const size_t plan = K::kWorkers * K::kWarp, smem = plan + (a.B <= kTableMost ? table_bytes(a.B) : 0);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_LAUNCH;
    if (!(prepared.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(plan + table_bytes(kTableMost))) != cudaSuccess) return FA_ERR_LAUNCH;
        prepared.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    // Twice the CTAs that one unit a worker takes, up to what the SMs hold.
    const long long items = (long long)a.Hkv * ((long long)a.T * a.G / K::kRows + (a.T < a.B ? a.T : a.B));
    const long long need = (items * ((((long long)a.W << a.ps_log2) + kUnit - 1) / kUnit + K::kExtra) + K::kWorkers - 1) / K::kWorkers;
    const int grid = 2 * need < sms ? (int)(2 * need) : sms;
    if (launch_dependent(kern, grid, K::kThreads, smem, stream, a) != cudaSuccess) return FA_ERR_LAUNCH;
    const long long rows = (long long)a.T * a.Hq;
    cudaError_t e;
    if (rows <= 8LL * sms) e = launch_dependent(kv4_join_kernel<D, true, K::kExtra>, (int)rows, 256, 0, stream, a, K::kRows);
    else e = launch_dependent(kv4_join_kernel<D, false, K::kExtra>, (int)((rows + 7) / 8), 256, 0, stream, a, K::kRows);
    return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}
template <int D, int NT> int launch_warps(const KvArgs& a, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> prepared{0};
    return launch_few<Kv<D, NT>, D>(kv4_kernel<D, NT>, prepared, a, sms, stream);
}
template <int D, int N> int launch_mid(const KvArgs& a, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> prepared{0};
    return launch_few<Mid<D, N>, D>(kv4_mid_kernel<D, N>, prepared, a, sms, stream);
}

int check_pages(int Hkv, int d, int num_pages, int page_size) {
    if (Hkv < 1 || d < 1 || num_pages < 1) return FA_ERR_INVALID;
    if ((d != 64 && d != 128 && d != 256) || page_log2(page_size) < 0) return FA_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_kv4_expand(const void* k_pages, const void* k_scales, const void* v_pages, const void* v_scales, const int* pages, int n,
                  int Hkv, int d, int num_pages, int page_size, void* k_out, void* v_out, cudaStream_t stream) {
    if (!k_pages || !k_scales || !v_pages || !v_scales || n < 0 || (n > 0 && (!k_out || !v_out))) return FA_ERR_INVALID;
    const int rc = check_pages(Hkv, d, num_pages, page_size);
    if (rc != FA_OK) return rc;
    if (!pages && n > num_pages) return FA_ERR_INVALID;
    if ((long long)n * Hkv > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    if (misaligned(k_pages, 15) || misaligned(v_pages, 15) || misaligned(k_scales, 15) || misaligned(v_scales, 15) || misaligned(k_out, 15) ||
        misaligned(v_out, 15) || misaligned(pages, 3))
        return FA_ERR_ALIGN;
    if (n == 0) return FA_OK;
    const size_t cells = (size_t)num_pages * Hkv * page_size, out = (size_t)n * Hkv * page_size * d * 2;
    const Span in[] = {{k_pages, cells * (d / 2)}, {v_pages, cells * (d / 2)}, {k_scales, cells * (d / 32)}, {v_scales, cells * (d / 32)},
                       {pages, pages ? 4 * (size_t)n : 0}};
    if (overlap({k_out, out}, {v_out, out})) return FA_ERR_INVALID;
    for (const Span& s : in)
        if (overlap({k_out, out}, s) || overlap({v_out, out}, s)) return FA_ERR_INVALID;
    const int sms = fa_num_sms();
    if (sms < 1) return FA_ERR_LAUNCH;
    const ExpandArgs a = {static_cast<const uint8_t*>(k_pages), static_cast<const uint8_t*>(k_scales), static_cast<const uint8_t*>(v_pages),
                          static_cast<const uint8_t*>(v_scales), static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out),
                          pages, nullptr, nullptr, n, 1, Hkv, num_pages, page_log2(page_size)};
    return launch_expand(a, d, sms, stream);
}

size_t fa_kv4_workspace_size(int T, int B, int Hq, int Hkv, int d, int max_seqlen, int table_width, int page_size) {
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 128 || max_seqlen < 1 || table_width < 1 ||
        (d != 64 && d != 128 && d != 256) || page_log2(page_size) < 0 || (long long)Hq * T > 0x7fffffffLL ||
        (long long)B * table_width > 0x7fffffffLL || (long long)table_width * page_size > kMaxKeys)
        return 0;
    const int sms = fa_num_sms();
    if (max_seqlen > T) max_seqlen = T > 1 ? T : 1;
    const size_t few = kv_layout(T, B, Hkv, Hq / Hkv, d, sms > 0 ? sms : kMaxSMs).total;
    const size_t many = many_layout(T, B, Hq, Hkv, d, max_seqlen, table_width, page_size).total;
    return few > many ? few : many;
}

int fa_kv4_fwd(const void* q, int64_t q_stride, const void* k_pages, const void* k_scales, const void* v_pages, const void* v_scales,
               void* o, float* lse, int T, int B, int Hq, int Hkv, int d, float alpha, int num_pages, int page_size,
               const int* block_table, int table_width, const int* kv_lens, const int* cu_seqlens, int max_seqlen, void* workspace,
               size_t workspace_bytes, cudaStream_t stream) {
    if (!q || !k_pages || !k_scales || !v_pages || !v_scales || !o || !lse || !block_table || !kv_lens) return FA_ERR_INVALID;
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_pages < 1 || table_width < 1 || max_seqlen < 1) return FA_ERR_INVALID;
    if (!(alpha > 0.0f) || !isfinite(alpha)) return FA_ERR_INVALID;
    if (!cu_seqlens && T != B) return FA_ERR_INVALID;
    if (q_stride < (long long)Hq * d) return FA_ERR_INVALID;
    const int rc = check_pages(Hkv, d, num_pages, page_size);
    if (rc != FA_OK) return rc;
    if (Hq / Hkv > 128 || B > kMaxVarlenSeqs) return FA_ERR_UNSUPPORTED;
    const long long lim = 0x7fffffffLL;
    if ((long long)Hq * T > lim || (long long)B * table_width > lim || (long long)table_width * page_size > kMaxKeys) return FA_ERR_UNSUPPORTED;
    if (misaligned(q, 15) || misaligned(k_pages, 15) || misaligned(v_pages, 15) || misaligned(k_scales, 15) || misaligned(v_scales, 15) ||
        misaligned(o, 15) || misaligned(lse, 15) || misaligned(block_table, 3) || misaligned(kv_lens, 3) || misaligned(cu_seqlens, 3) || (q_stride & 7))
        return FA_ERR_ALIGN;
    if (T == 0) return FA_OK;
    const int G = Hq / Hkv;
    if (max_seqlen > T) max_seqlen = T;
    // The list of units at its longest fits 32 bits, a worker's share past it too.
    const long long tiles = ((long long)table_width * page_size + kUnit - 1) / kUnit + kExtraMost;
    const long long items = (long long)Hkv * ((long long)T * G / 8 + (T < B ? T : B));
    if (items * (tiles + 1) > 1 << 30) return FA_ERR_UNSUPPORTED;
    const size_t row = (size_t)Hq * d * 2, cells = (size_t)num_pages * Hkv * page_size;
    const Span inputs[] = {{k_pages, cells * (d / 2)}, {v_pages, cells * (d / 2)}, {k_scales, cells * (d / 32)}, {v_scales, cells * (d / 32)},
                           {block_table, 4 * (size_t)B * table_width}, {kv_lens, 4 * (size_t)B}, {cu_seqlens, cu_seqlens ? 4 * ((size_t)B + 1) : 0}};
    auto over_input = [&](const Span& out) {
        for (const Span& in : inputs)
            if (overlap(out, in)) return true;
        return overlap_rows(out, q, T, row, (size_t)q_stride * 2);
    };
    const Span out_o = {o, T * row}, out_lse = {lse, 4 * (size_t)Hq * T};
    if (over_input(out_o) || over_input(out_lse) || overlap(out_o, out_lse)) return FA_ERR_INVALID;
    const int sms = fa_num_sms();
    DevStatus* status = device_status_ptr();
    if (sms < 1 || !status) return FA_ERR_LAUNCH;
    const KvLayout w = kv_layout(T, B, Hkv, G, d, sms);
    const ManyLayout many = many_layout(T, B, Hq, Hkv, d, max_seqlen, table_width, page_size);
    if (!workspace || misaligned(workspace, 255) || workspace_bytes < w.total) return FA_ERR_WORKSPACE;
    const bool expand = many.total > 0 && workspace_bytes >= many.total;
    const Span scratch = {workspace, expand ? many.total : w.total};
    if (over_input(scratch) || overlap(scratch, out_o) || overlap(scratch, out_lse)) return FA_ERR_INVALID;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const uint8_t *kp = static_cast<const uint8_t*>(k_pages), *ks = static_cast<const uint8_t*>(k_scales),
                  *vp = static_cast<const uint8_t*>(v_pages), *vs = static_cast<const uint8_t*>(v_scales);
    const int lg = page_log2(page_size);
    if (expand) {
        int* table = reinterpret_cast<int*>(ws + many.table);
        const ExpandArgs e = {kp, ks, vp, vs, reinterpret_cast<__nv_bfloat16*>(ws), reinterpret_cast<__nv_bfloat16*>(ws + many.v),
                              block_table, kv_lens, table, B * table_width, table_width, Hkv, num_pages, lg};
        const int rc2 = launch_expand(e, d, sms, stream);
        if (rc2 != FA_OK) return rc2;
        return fa_prefix_fwd(q, q_stride, ws, ws + many.v, o, lse, T, B, Hq, Hkv, d, alpha, B * table_width, page_size, table, table_width,
                             kv_lens, cu_seqlens, max_seqlen, nullptr, 0, ws + many.prefix, many.total - many.prefix, stream);
    }
    KvArgs a;
    a.kp = kp;
    a.ks = ks;
    a.vp = vp;
    a.vs = vs;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.table = block_table;
    a.kv_lens = kv_lens;
    a.cu = cu_seqlens;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.status = status;
    a.hdr = reinterpret_cast<KvHeader*>(ws);
    a.tables = reinterpret_cast<int*>(ws + w.tables);
    a.rows = reinterpret_cast<KvRow*>(ws + w.rows);
    a.ml = reinterpret_cast<float2*>(ws + w.ml);
    a.seg = reinterpret_cast<float*>(ws + w.seg);
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.W = table_width;
    a.P = num_pages;
    a.ps_log2 = lg;
    a.max_seqlen = max_seqlen;
    a.scale_log2 = alpha * 1.4426950408889634f;
    // Which kernel, by rows an item: see the figures at "more rows".
    const int rows = item_rows(max_seqlen * (long long)G);
    if (d == 64) return rows == 8 ? launch_warps<64, 1>(a, sms, stream) : rows == 16 ? launch_warps<64, 2>(a, sms, stream) : launch_mid<64, 32>(a, sms, stream);
    if (d == 128) return rows == 8 ? launch_warps<128, 1>(a, sms, stream) : rows == 16 ? launch_warps<128, 2>(a, sms, stream) : launch_mid<128, 32>(a, sms, stream);
    return rows == 8 ? launch_warps<256, 1>(a, sms, stream) : rows == 16 ? launch_mid<256, 16>(a, sms, stream) : launch_mid<256, 32>(a, sms, stream);
}

}  // extern "C"

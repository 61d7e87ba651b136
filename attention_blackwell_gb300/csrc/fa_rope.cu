// fa_rope.cu -- what lies between the projections and attention (sm_103a):
// fa_qk_rope (norms per head and position rotation of Q and K), fa_qk_rope_bwd
// (their gradients) and fa_rope_store (the same on the way into a paged cache of
// bf16 or 4-bit rows).
//
//   n(x) = x r w, r = (mean x^2 + eps)^(-1/2)   over a head's d elements, or x
//   y = R n(x): the first rot elements in pairs (i, i + rot/2) or (2i, 2i + 1),
//       (a, b) -> (a cos - b sin, b cos + a sin), the angles of the token's position
// and, for u = R^T dy and t = u w,
//   dx = r (t - x r^2 mean(t x)),   dw = sum over rows of u x r.
// All of it in 32 bits, rounded once where it is stored.
//
// A unit is up to r.chunk rows of one token's q, k or v, which are adjacent in memory,
// with its rows of the cos and sin tables.  Every warp has a ring of units in shared
// memory, filled by bulk copies (what is in flight costs no registers; loaded into
// registers ahead, the same work moved 5.0 TB/s at its best), and takes a range of
// the call's units.  d / 16 lanes share a row, so that a lane's 16 elements are
// whole pairs whatever rot is: two 16-byte chunks.
//
// What bounds them (GB300; 6.78 TB/s measured, times of calls back to back): HBM,
// after a start of 4 us (positions, then tables and rows).  16384 tokens of 16 + 16
// heads of 128 with norms: forward 46 us (271 MB, 5.9 TB/s), gradients 70 (405 MB; 5 of
// them the sum over blocks).  10003 tokens of 8 + 1 heads of 256: gradients 39 (139 MB):
// a unit of one row, k's, costs half of one of eight.  20011 tokens of 32 + 8 + 8 heads
// into a 4-bit cache: 73 (432 MB), 2730 instructions a token, 65 % of the issue
// slots.  64 tokens: 4 us on the GPU; the call from Python takes 13 to 18.
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_kv4.cuh"

namespace fa {
namespace {

// What a call rotates and how.
struct RopeArgs {
    const float *cos, *sin;      // [max_pos, rot / 2]
    const int* positions;        // [T] or null: t % seq_len
    const void *wq, *wk;         // [d] float or bf16, null: no norm
    int T, Hq, Hkv, max_pos, rot, inter, seq_len, w_bf16;
    float eps;
    int chunk, per_q, per_k, per;    // rows a unit; units of a token's q rows, of its k (and v) rows, of all
    int units;
    int clear;                   // bits 0 and 1: q's, k's outputs of tokens off the tables become 0
    DevStatus* status;
};

struct RowsArgs {
    const __nv_bfloat16 *q, *k;
    __nv_bfloat16 *q_out, *k_out;
    long long q_stride, k_stride, q_out_stride, k_out_stride;
};

struct GradArgs {
    const __nv_bfloat16 *gq, *gk, *q, *k;
    __nv_bfloat16 *dq, *dk;
    long long gq_stride, gk_stride, q_stride, k_stride;
    float* partial;              // [grid][2][d]
};

struct PutArgs {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* q_out;
    long long q_stride, k_stride, v_stride, q_out_stride;
    const int* slots;
    uint8_t *kp, *vp, *ks, *vs;  // pages and, with 4 bits, their scales
    int ps_log2;
    long long num_slots;
};

// Two floats in a register pair: products and sums of a row's elements go two an
// instruction (as one each, qk_rope spent half as much again on arithmetic).
using F2 = uint64_t;
__device__ __forceinline__ F2 both(float x) { return f2_pack(x, x); }

// The lane's place in a row and its angles.
template <int D> struct Lane {
    static constexpr int kLanes = D / 16, kRows = 32 / kLanes;   // lanes a row, rows a pass
    int a, b;            // first elements of its two chunks of eight
    bool turns;
    F2 c[4], s[4], ns[4];    // ns = -s
    __device__ __forceinline__ void place(const RopeArgs& r, int lane) {
        const int j = lane % kLanes, m = r.rot >> 4;
        turns = j < m;
        const bool split = turns && !r.inter;
        a = (split ? j : 2 * j) * 8;
        b = (split ? j + m : 2 * j + 1) * 8;
    }
    // From the unit's rows of the tables; sign -1: the angles' opposites.
    template <bool kWhole> __device__ __forceinline__ void angles(const RopeArgs& r, const float* table, int lane, float sign) {
        if (!kWhole && !turns) return;
        const float4 *pc = reinterpret_cast<const float4*>(table + lane % kLanes * 8), *ps = reinterpret_cast<const float4*>(table + (r.rot >> 1) + lane % kLanes * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = pc[i], y = ps[i];
            c[2 * i] = f2_pack(x.x, x.y), c[2 * i + 1] = f2_pack(x.z, x.w);
            s[2 * i] = f2_pack(sign * y.x, sign * y.y), s[2 * i + 1] = f2_pack(sign * y.z, sign * y.w);
            ns[2 * i] = f2_pack(-sign * y.x, -sign * y.y), ns[2 * i + 1] = f2_pack(-sign * y.z, -sign * y.w);
        }
    }
    // kWhole: all of a row, in halves, without a branch: a store into 4-bit pages, which
    // is bound by its instructions, gains 5 % (20011 tokens stored and expanded 96 us, 91
    // so); qk_rope, which HBM binds, gains nothing.
    template <bool kWhole> __device__ __forceinline__ void turn(F2 (&v)[8], bool inter) const {
        if (!kWhole && !turns) return;
        if (kWhole || !inter) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F2 x = v[i], y = v[4 + i];
                v[i] = f2_fma(y, ns[i], f2_mul(x, c[i]));
                v[4 + i] = f2_fma(x, s[i], f2_mul(y, c[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float c0, c1, s0, s1, x0, y0, x1, y1;
                f2_unpack(c[i], c0, c1);
                f2_unpack(s[i], s0, s1);
                f2_unpack(v[2 * i], x0, y0);
                f2_unpack(v[2 * i + 1], x1, y1);
                v[2 * i] = f2_pack(x0 * c0 - y0 * s0, y0 * c0 + x0 * s0);
                v[2 * i + 1] = f2_pack(x1 * c1 - y1 * s1, y1 * c1 + x1 * s1);
            }
        }
    }
};

__device__ __forceinline__ int position_of(const RopeArgs& r, int t) {
    const int p = r.positions ? r.positions[t] : t % r.seq_len;
    return p >= 0 && p < r.max_pos ? p : -1;
}

__device__ __forceinline__ void unpack8(const uint4& u, F2* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(F2 v) {
    float x, y;
    f2_unpack(v, x, y);
    return pack_bf16x2(x, y);
}
__device__ __forceinline__ uint4 pack8(const F2* v) { return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])); }
__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Sum over the lanes of a row.
template <int L> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float sum2(F2 v) {
    float x, y;
    f2_unpack(v, x, y);
    return x + y;
}
template <int D> __device__ __forceinline__ float inv_rms(const F2 (&v)[8], float eps) {
    F2 s0 = f2_mul(v[0], v[0]), s1 = f2_mul(v[1], v[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s0 = f2_fma(v[i], v[i], s0);
        s1 = f2_fma(v[i + 1], v[i + 1], s1);
    }
    return rsqrtf(row_sum<D / 16>(sum2(f2_add(s0, s1))) * (1.f / D) + eps);
}

// Both weights in shared memory as floats ([2][D]; rows of 1 for the one without a norm).
template <int D> __device__ __forceinline__ void stage_weights(const RopeArgs& r, float* w) {
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const void* src = i < D ? r.wq : r.wk;
        const int e = i & (D - 1);
        w[i] = !src ? 1.f : r.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(src)[e]) : static_cast<const float*>(src)[e];
    }
}
// The lane's weights (w: a row of D).
template <int D> __device__ __forceinline__ void weights_of(const float* w, const Lane<D>& me, F2 (&out)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(w + me.a + 4 * i), y = *reinterpret_cast<const ulonglong2*>(w + me.b + 4 * i);
        out[2 * i] = x.x, out[2 * i + 1] = x.y;
        out[4 + 2 * i] = y.x, out[4 + 2 * i + 1] = y.y;
    }
}
template <int D> __device__ __forceinline__ void weigh(F2 (&v)[8], float x, const float* w, const Lane<D>& me) {
    F2 ww[8];
    weights_of<D>(w, me, ww);
    const F2 xx = both(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f2_mul(f2_mul(v[i], xx), ww[i]);
}

// ------------------------------------------------------------------ the units

// What a unit is, at the head of its slot.
struct __align__(16) Unit {
    int t, j, pos, slot;     // token, unit of the token, position, slot of the cache
};

// A warp's ring of units: kArrays arrays of kBytes (the rows), the tables' rows.
template <int D, int kBytes, int kArrays, int kRing> struct Feed {
    static constexpr uint32_t kTable = 16 + kArrays * kBytes, kSlot = kTable + D * 4, kWarp = kRing * kSlot;
    static_assert(kSlot % 16 == 0 && kRing <= 4, "copies are 16-byte aligned");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Calls work(unit, rows, tables) for this warp's units.  rows(t, j, array, bytes) is
// where a unit's rows are and how many bytes of them; off(t, j) is called for those of
// tokens off the tables, which are passed over, where something becomes of them.
template <int D, int kBytes, int kArrays, int kRing, int kWarps, class Rows, class Off, class Work>
__device__ __forceinline__ void feed(const RopeArgs& r, uint8_t* ring, uint64_t* full, const int* slots, const Rows& rows, const Off& off, const Work& work) {
    using F = Feed<D, kBytes, kArrays, kRing>;
    const int lane = threadIdx.x & 31;
    // A range of the units, so that every warp gets q, k and v in the same proportion.
    const int warps = gridDim.x * kWarps, warp = blockIdx.x * kWarps + (threadIdx.x >> 5), share = r.units / warps, more = r.units - share * warps;
    const int first = warp * share + min(warp, more), n = share + (warp < more);
    // The units that the copies come to next, 32 at a time, one a lane, and the 32 after them.
    auto fetch = [&](int k) {
        Unit u = {0, 0, -1, 0};
        if (k + lane < n) {
            const int id = first + k + lane;
            u.t = id / r.per;
            u.j = id - u.t * r.per;
            u.pos = position_of(r, u.t);
            u.slot = slots ? slots[u.t] : 0;
        }
        return u;
    };
    Unit now = fetch(0), next = fetch(32);
    int k = 0;
    uint32_t filled = 0, issued = 0;
    auto copy = [&]() {
        Unit u;
        for (;;) {
            if (k >= n) return;
            if (k && (k & 31) == 0) {
                now = next;
                next = fetch(k + 32);
            }
            const int i = k & 31;
            u.pos = __shfl_sync(0xffffffffu, now.pos, i);
            u.t = __shfl_sync(0xffffffffu, now.t, i);
            u.j = __shfl_sync(0xffffffffu, now.j, i);
            u.slot = __shfl_sync(0xffffffffu, now.slot, i);
            ++k;
            if (u.pos >= 0) break;
            if (r.clear) off(u.t, u.j);
        }
        uint8_t* to = ring + filled * F::kSlot;
        uint64_t* bar = &full[filled];
        uint32_t bytes = r.rot * 2, total = 2 * bytes;
        const uint8_t* from;
        if (lane < kArrays) from = rows(u.t, u.j, lane, bytes);
        else from = reinterpret_cast<const uint8_t*>((lane == kArrays ? r.cos : r.sin) + (long long)u.pos * (r.rot >> 1));
#pragma unroll
        for (int i = 0; i < kArrays; ++i) total += __shfl_sync(0xffffffffu, bytes, i);
        __syncwarp();                                // every lane has read what the slot held
        if (lane == 0) {
            *reinterpret_cast<Unit*>(to) = u;
            mbar_arrive_expect_tx(bar, total);
        }
        __syncwarp();
        if (lane < kArrays + 2 && bytes) bulk_load(smem_u32(to) + (lane < kArrays ? 16 + lane * kBytes : F::kTable + (lane - kArrays) * r.rot * 2), from, bytes, bar);
        filled = filled + 1 == kRing ? 0 : filled + 1;
        ++issued;
    };
    for (int i = 0; i < kRing; ++i) copy();
    uint32_t slot = 0, phase = 0;
    for (uint32_t done = 0; done != issued; ++done) {
        // The bounded wait (2 s); after one that gave up, the copies in flight get as long again.
        const uint32_t bar = smem_u32(&full[slot]);
        bool ok = mbar_try_wait(bar, phase);
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            while (!(ok = mbar_try_wait(bar, phase)) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
        if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0 && atomicCAS(&r.status->code, 0, kStatusTimeout) == 0) {
                r.status->where = 121;
                r.status->block = blockIdx.x;
            }
            const uint64_t t0 = globaltimer_ns();
            for (; done != issued; ++done) {
                while (!mbar_try_wait(smem_u32(&full[slot]), phase) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                if (++slot == kRing) slot = 0, phase ^= 1;
            }
            return;
        }
        const uint8_t* at = ring + slot * F::kSlot;
        work(*reinterpret_cast<const Unit*>(at), at + 16, reinterpret_cast<const float*>(at + F::kTable));
        if (++slot == kRing) slot = 0, phase ^= 1;
        __syncwarp();
        copy();
    }
}

// Which rows of a token unit j is: of q (0), k (1) or v (2), from row h0 on, n of them.
struct Chunk {
    int what, h0, n;
};
__device__ __forceinline__ Chunk chunk_of(const RopeArgs& r, int j) {
    Chunk c;
    c.what = j < r.per_q ? 0 : j < r.per_q + r.per_k ? 1 : 2;
    c.h0 = (c.what == 0 ? j : c.what == 1 ? j - r.per_q : j - r.per_q - r.per_k) * r.chunk;
    c.n = min(r.chunk, (c.what == 0 ? r.Hq : r.Hkv) - c.h0);
    return c;
}

// A unit's rows of an output as 0, if it is one that the call clears.
template <int D> __device__ __forceinline__ void clear_rows(const RopeArgs& r, const Chunk& c, __nv_bfloat16* token) {
    if (!(r.clear >> (c.what != 0) & 1)) return;
    uint4* to = reinterpret_cast<uint4*>(token + c.h0 * D);
    for (int i = threadIdx.x & 31; i < c.n * (D / 8); i += 32) to[i] = make_uint4(0, 0, 0, 0);
}

// Bytes of rows a unit at most, of each array: four passes of 32 lanes.  What a unit
// costs besides its passes is worth one of them.
constexpr int kBytes = 4096, kBytesGrad = 4096, kRing = 3, kRingPut = 2, kRingGrad = 2;
constexpr int kWarps = 12, kWarpsPut = 16, kWarpsGrad = 12;      // a block, one an SM
template <int D> constexpr int kPass = 512 / D;              // rows a pass
template <int D> constexpr int kChunk = kBytes / (2 * D);
template <int D> constexpr int kChunkGrad = kBytesGrad / (2 * D);
template <int D> constexpr uint32_t kSmem = kWarps * Feed<D, kBytes, 1, kRing>::kWarp;
template <int D> constexpr uint32_t kSmemPut = kWarpsPut * Feed<D, kBytes, 1, kRingPut>::kWarp;
template <int D> constexpr uint32_t kSmemGrad = kWarpsGrad * Feed<D, kBytesGrad, 2, kRingGrad>::kWarp;

// The block's barriers, before the kernel it depends on is done.
template <int W, int N> __device__ __forceinline__ void init_barriers(uint64_t (&full)[W][N]) {
    if (threadIdx.x < W * N) {
        mbar_init(&full[0][0] + threadIdx.x, 1);
        fence_mbar_init();
    }
}

// ------------------------------------------------------------------ forward

// A unit's rows of q or k, normed and turned, to out(row).
template <int D, bool kWhole, class Out>
__device__ __forceinline__ void turn_rows(const RopeArgs& r, Lane<D>& me, const Chunk& c, const uint8_t* in, const float* table, const float* s_w, const Out& out) {
    using Me = Lane<D>;
    const int lane = threadIdx.x & 31, sub = lane / Me::kLanes;
    const bool norm = c.what ? r.wk != nullptr : r.wq != nullptr;
    me.template angles<kWhole>(r, table, lane, 1.f);
    auto pass = [&](int p, bool real) {
        const int i = p + sub;
        F2 v[8] = {};
        if (real) {
            unpack8(load16(in + (i * D + me.a) * 2), v);
            unpack8(load16(in + (i * D + me.b) * 2), v + 4);
        }
        if (norm) weigh<D>(v, inv_rms<D>(v, r.eps), s_w + (c.what ? D : 0), me);
        me.template turn<kWhole>(v, r.inter);
        if (real) {
            __nv_bfloat16* dst = out(c.h0 + i);
            *reinterpret_cast<uint4*>(dst + me.a) = pack8(v);
            *reinterpret_cast<uint4*>(dst + me.b) = pack8(v + 4);
        }
    };
#pragma unroll (kWhole ? 1 : kChunk<D> / Me::kRows)
    for (int p = 0; p < kChunk<D>; p += Me::kRows) {
        if (p >= c.n) break;
        pass(p, p + sub < c.n);
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 1) qk_rope_kernel(const RopeArgs r, const RowsArgs a) {
    extern __shared__ __align__(16) uint8_t dsmem[];
    __shared__ __align__(16) float s_w[2 * D];
    __shared__ uint64_t full[kWarps][kRing];
    init_barriers(full);
    grid_launch_next();
    grid_wait();
    if (r.wq || r.wk) stage_weights<D>(r, s_w);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Lane<D> me;
    me.place(r, lane);
    auto rows = [&](int t, int j, int, uint32_t& bytes) {
        const Chunk c = chunk_of(r, j);
        bytes = c.n * D * 2;
        return reinterpret_cast<const uint8_t*>((c.what ? a.k + t * a.k_stride : a.q + t * a.q_stride) + c.h0 * D);
    };
    auto out = [&](int t, const Chunk& c) { return c.what ? a.k_out + t * a.k_out_stride : a.q_out + t * a.q_out_stride; };
    auto off = [&](int t, int j) {
        const Chunk c = chunk_of(r, j);
        clear_rows<D>(r, c, out(t, c));
    };
    feed<D, kBytes, 1, kRing, kWarps>(r, dsmem + warp * Feed<D, kBytes, 1, kRing>::kWarp, full[warp], nullptr, rows, off,
                              [&](const Unit& u, const uint8_t* in, const float* table) {
        const Chunk c = chunk_of(r, u.j);
        __nv_bfloat16* to = out(u.t, c);
        turn_rows<D, false>(r, me, c, in, table, s_w, [&](int h) { return to + h * D; });
    });
}

// ----------------------------------------------------------------- gradients

// A pass over rows of q or k; dw: the lane's share of the weight's gradient.
template <int D>
__device__ __forceinline__ void grad_row(const RopeArgs& r, const Lane<D>& me, bool real, const uint8_t* g, const uint8_t* x, const float* w, F2 (&dw)[8], __nv_bfloat16* out) {
    F2 u[8] = {};
    if (real) {
        unpack8(load16(g + me.a * 2), u);
        unpack8(load16(g + me.b * 2), u + 4);
    }
    me.template turn<false>(u, r.inter);
    if (w) {
        F2 v[8] = {};
        if (real) {
            unpack8(load16(x + me.a * 2), v);
            unpack8(load16(x + me.b * 2), v + 4);
        }
        // With eps = 0 a missing row's r is infinite.
        const float rms = inv_rms<D>(v, r.eps), x1 = real ? rms : 0.f;
        const F2 xx = both(x1);
        F2 ww[8], sum = 0;
        weights_of<D>(w, me, ww);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = f2_mul(v[e], xx);                        // x r
            dw[e] = f2_fma(u[e], v[e], dw[e]);
            u[e] = f2_mul(u[e], ww[e]);
            sum = f2_fma(u[e], v[e], sum);
        }
        const F2 mean = both(row_sum<D / 16>(sum2(sum)) * (-1.f / D));      // -mean(t x) r
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = f2_mul(f2_fma(v[e], mean, u[e]), xx);
    }
    if (real) {
        *reinterpret_cast<uint4*>(out + me.a) = pack8(u);
        *reinterpret_cast<uint4*>(out + me.b) = pack8(u + 4);
    }
}

// Each block leaves its sums of the weights' gradients, which a second kernel adds up
// in the blocks' order, so equal calls give equal results.
template <int D>
__global__ void __launch_bounds__(32 * kWarpsGrad, 1) qk_rope_bwd_kernel(const RopeArgs r, const GradArgs a) {
    using Me = Lane<D>;
    extern __shared__ __align__(16) uint8_t dsmem[];
    __shared__ __align__(16) float s_w[2 * D];
    __shared__ uint64_t full[kWarpsGrad][kRingGrad];
    init_barriers(full);
    grid_launch_next();
    grid_wait();
    const bool norm = r.wq || r.wk;
    if (norm) stage_weights<D>(r, s_w);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / Me::kLanes;
    Me me;
    me.place(r, lane);
    F2 dwq[8] = {}, dwk[8] = {};
    auto rows = [&](int t, int j, int array, uint32_t& bytes) {
        const Chunk c = chunk_of(r, j);
        bytes = array && !(c.what ? r.wk : r.wq) ? 0 : c.n * D * 2;
        const __nv_bfloat16* p = c.what ? (array ? a.k + t * a.k_stride : a.gk + t * a.gk_stride) : array ? a.q + t * a.q_stride : a.gq + t * a.gq_stride;
        return reinterpret_cast<const uint8_t*>(p + c.h0 * D);
    };
    auto token = [&](int t, const Chunk& c) { return c.what ? a.dk + (long long)t * r.Hkv * D : a.dq + (long long)t * r.Hq * D; };
    auto off = [&](int t, int j) {
        const Chunk c = chunk_of(r, j);
        clear_rows<D>(r, c, token(t, c));
    };
    feed<D, kBytesGrad, 2, kRingGrad, kWarpsGrad>(r, dsmem + warp * Feed<D, kBytesGrad, 2, kRingGrad>::kWarp, full[warp], nullptr, rows, off,
                                  [&](const Unit& u, const uint8_t* in, const float* table) {
        const Chunk c = chunk_of(r, u.j);
        me.template angles<false>(r, table, lane, -1.f);
        __nv_bfloat16* out = token(u.t, c) + c.h0 * D;
        const uint8_t* g = in + sub * D * 2;
        auto passes = [&](const float* w, F2 (&dw)[8]) {
            for (int p = 0; p < c.n; p += Me::kRows)
                grad_row<D>(r, me, p + sub < c.n, g + p * D * 2, g + p * D * 2 + kBytesGrad, w, dw, out + (p + sub) * D);
        };
        if (c.what == 0) passes(r.wq ? s_w : nullptr, dwq);
        else passes(r.wk ? s_w + D : nullptr, dwk);
    });
    if (!norm) return;
    // The warp's rows, then the block's warps; the rings are done with.
    __syncthreads();
    float (*s_dw)[2 * D] = reinterpret_cast<float (*)[2 * D]>(dsmem);
    static_assert(kWarpsGrad * 2 * D * 4 <= kSmemGrad<D>, "room for the sums");
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float q[2], k[2];
        f2_unpack(dwq[e >> 1], q[0], q[1]);
        f2_unpack(dwk[e >> 1], k[0], k[1]);
        float x = q[e & 1], y = k[e & 1];
#pragma unroll
        for (int o = 16; o >= Me::kLanes; o >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, o);
            y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        if (sub == 0) {
            const int i = (e < 8 ? me.a : me.b - 8) + e;
            s_dw[warp][i] = x;
            s_dw[warp][D + i] = y;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarpsGrad) {
        float sum = s_dw[0][i];
#pragma unroll
        for (int y = 1; y < kWarpsGrad; ++y) sum += s_dw[y][i];
        a.partial[(long long)blockIdx.x * (2 * D) + i] = sum;
    }
}

// 32 columns of the blocks' sums a block, 32 rows at a time.
__global__ void __launch_bounds__(1024) qk_rope_dw_kernel(const float* partial, int blocks, int d, float* dwq, float* dwk) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
    grid_wait();
    float sum = 0.f;
    for (int b = y; b < blocks; b += 32) sum += partial[(long long)b * (2 * d) + col];
    s[y][x] = sum;
    __syncthreads();
    // A column a warp, its 32 sums a lane each, in one order.
    sum = s[x][y];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int at = blockIdx.x * 32 + y;
    float* out = at < d ? dwq : dwk;
    if (x == 0 && out) out[at & (d - 1)] = sum;
}

// --------------------------------------------------------------------- store

__device__ __forceinline__ float max_abs(float a, float b) {     // NaN if either is; the sign means nothing
    float m;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Eight lanes' row y (lane l: elements 32 g + 4 l to + 3) as 4-bit codes and scales
// (see fa_kv4.cuh).  A group's scale is worked out by one lane for all eight.
template <int D>
__device__ __forceinline__ void put_codes(const F2 (&y)[D / 32][2], bool real, uint8_t* codes, uint8_t* scales, int lane) {
    constexpr int kG = D / 32;
    const int l = lane & 7;
    uint32_t most[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        float a, b, c, d;
        f2_unpack(y[g][0], a, b);
        f2_unpack(y[g][1], c, d);
        most[g] = __float_as_uint(max_abs(max_abs(a, b), max_abs(c, d))) & 0x7fffffffu;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
        for (int g = 0; g < kG; ++g) most[g] = max(most[g], __shfl_xor_sync(0xffffffffu, most[g], o));
    uint32_t mine = most[0];
#pragma unroll
    for (int g = 1; g < kG; ++g) mine = l % kG == g ? most[g] : mine;
    const uint32_t byte = scale_byte(mine);
    const bool plain = byte != 0 && byte != kScaleNaN;       // else codes of 0
    const float minus_s = plain ? -scale_f32(byte) : 0.f, inv_own = plain ? __frcp_rn(-minus_s) : 0.f;
    uint32_t out[kG / 2];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        const F2 s = both(__shfl_sync(0xffffffffu, minus_s, (lane & 24) + g)), inv = both(__shfl_sync(0xffffffffu, inv_own, (lane & 24) + g));
        const uint32_t c = codes_of(y[g][0], y[g][1], s, inv);
        out[g / 2] = g & 1 ? out[g / 2] | c << 16 : c;
    }
    if (!real) return;
    uint32_t* dst = reinterpret_cast<uint32_t*>(codes) + l * (kG / 2);
    if constexpr (D == 64) *dst = out[0];
    else if constexpr (D == 128) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    if (l < kG) scales[l] = (uint8_t)byte;
}

__device__ __forceinline__ void unpack4(const uint2& u, F2 (&y)[2]) {
    y[0] = f2_pack(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    y[1] = f2_pack(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// A row by eight lanes, normed where there are weights.
template <int D>
__device__ __forceinline__ void norm_four(const RopeArgs& r, const uint8_t* row, bool norm, const float* w, int l, F2 (&y)[D / 32][2], float& x) {
    constexpr int kG = D / 32;
#pragma unroll
    for (int g = 0; g < kG; ++g) unpack4(*reinterpret_cast<const uint2*>(row + (32 * g + 4 * l) * 2), y[g]);
    if (!norm) return;
    F2 sum = 0;
#pragma unroll
    for (int g = 0; g < kG; ++g) sum = f2_fma(y[g][1], y[g][1], f2_fma(y[g][0], y[g][0], sum));
    x = rsqrtf(row_sum<8>(sum2(sum)) * (1.f / D) + r.eps);
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        const ulonglong2 ww = *reinterpret_cast<const ulonglong2*>(w + 32 * g + 4 * l);
        y[g][0] = f2_mul(f2_mul(y[g][0], both(x)), ww.x);
        y[g][1] = f2_mul(f2_mul(y[g][1], both(x)), ww.y);
    }
}

// The rotation of a row that eight lanes hold.  Every product and sum is rounded by
// itself, as the formula reads: codes lie next to borders, and so it is plain which
// side a key falls on.  (One float an instruction: the compiler joins a product of
// two with the sum that follows.)  Whole rows in halves (the common case): a pair's two
// elements are the same lane's, d / 2 apart, and the angles stay in registers.
template <int D> struct Four {
    static constexpr int kG = D / 32;
    F2 c[kG / 2][2], s[kG / 2][2];
    const float *pc, *ps;    // the unit's rows of the tables
    __device__ __forceinline__ void angles(const RopeArgs& r, const float* table, int l, bool whole) {
        pc = table;
        ps = table + (r.rot >> 1);
        if (!whole) return;
#pragma unroll
        for (int g = 0; g < kG / 2; ++g) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(pc + 32 * g + 4 * l), y = *reinterpret_cast<const ulonglong2*>(ps + 32 * g + 4 * l);
            c[g][0] = x.x, c[g][1] = x.y;
            s[g][0] = y.x, s[g][1] = y.y;
        }
    }
    __device__ __forceinline__ void turn_whole(F2 (&y)[kG][2]) const {
#pragma unroll
        for (int g = 0; g < kG / 2; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a[2], b[2], cc[2], ss[2];
                f2_unpack(y[g][i], a[0], a[1]);
                f2_unpack(y[g + kG / 2][i], b[0], b[1]);
                f2_unpack(c[g][i], cc[0], cc[1]);
                f2_unpack(s[g][i], ss[0], ss[1]);
                float lo[2], hi[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    lo[e] = __fsub_rn(__fmul_rn(a[e], cc[e]), __fmul_rn(b[e], ss[e]));
                    hi[e] = __fadd_rn(__fmul_rn(b[e], cc[e]), __fmul_rn(a[e], ss[e]));
                }
                y[g][i] = f2_pack(lo[0], lo[1]);
                y[g + kG / 2][i] = f2_pack(hi[0], hi[1]);
            }
    }
    // Any other rotation: partners are read again.
    __device__ __forceinline__ void turn(const RopeArgs& r, const uint8_t* row, float x, const float* w, int l, F2 (&y)[kG][2]) const {
        const int half = r.rot >> 1;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            const int i = 32 * g + 4 * l;
            if (i >= r.rot) continue;
            float v[4];
            f2_unpack(y[g][0], v[0], v[1]);
            f2_unpack(y[g][1], v[2], v[3]);
            if (r.inter) {
                const float2 c2 = *reinterpret_cast<const float2*>(pc + (i >> 1)), s2 = *reinterpret_cast<const float2*>(ps + (i >> 1));
                y[g][0] = f2_pack(__fsub_rn(__fmul_rn(v[0], c2.x), __fmul_rn(v[1], s2.x)), __fadd_rn(__fmul_rn(v[1], c2.x), __fmul_rn(v[0], s2.x)));
                y[g][1] = f2_pack(__fsub_rn(__fmul_rn(v[2], c2.y), __fmul_rn(v[3], s2.y)), __fadd_rn(__fmul_rn(v[3], c2.y), __fmul_rn(v[2], s2.y)));
                continue;
            }
            const bool low = i < half;
            const int at = low ? i : i - half, there = low ? i + half : i - half;
            F2 z2[2];
            unpack4(*reinterpret_cast<const uint2*>(row + there * 2), z2);
            float z[4];
            f2_unpack(z2[0], z[0], z[1]);
            f2_unpack(z2[1], z[2], z[3]);
            const float4 c4 = *reinterpret_cast<const float4*>(pc + at), s4 = *reinterpret_cast<const float4*>(ps + at);
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (w) z[e] = z[e] * x * w[there + e];
                const float own = __fmul_rn(v[e], cc[e]), other = __fmul_rn(z[e], ss[e]);
                v[e] = low ? __fsub_rn(own, other) : __fadd_rn(own, other);
            }
            y[g][0] = f2_pack(v[0], v[1]);
            y[g][1] = f2_pack(v[2], v[3]);
        }
    }
};

// Rows of k or v into 4-bit pages, four rows a pass.
template <int D, bool kWhole>
__device__ __forceinline__ void put_rows(const RopeArgs& r, const PutArgs& a, const Chunk& c, const uint8_t* in, const float* table, const float* s_w, long long cell) {
    const int lane = threadIdx.x & 31, l = lane & 7;
    const bool isk = c.what == 1, norm = isk && r.wk != nullptr;
    const float* w = s_w + D;
    Four<D> turner;
    if (isk) turner.angles(r, table, l, kWhole);
#pragma unroll 1
    for (int i = lane >> 3; i - (lane >> 3) < c.n; i += 4) {
        const bool real = i < c.n;
        const uint8_t* row = in + (real ? i : 0) * (D * 2);
        F2 y[D / 32][2];
        float x = 1.f;
        norm_four<D>(r, row, norm, w, l, y, x);
        if (isk) {
            if (kWhole) turner.turn_whole(y);
            else turner.turn(r, row, x, norm ? w : nullptr, l, y);
        }
        const long long at = cell + ((long long)(c.h0 + i) << a.ps_log2);
        put_codes<D>(y, real, (isk ? a.kp : a.vp) + at * (D / 2), (isk ? a.ks : a.vs) + at * (D / 32), lane);
    }
}

template <int D, bool kFour, bool kWhole>
__global__ void __launch_bounds__(32 * kWarpsPut, 1) rope_store_kernel(const RopeArgs r, const PutArgs a) {
    using Me = Lane<D>;
    extern __shared__ __align__(16) uint8_t dsmem[];
    __shared__ __align__(16) float s_w[2 * D];
    __shared__ uint64_t full[kWarpsPut][kRingPut];
    init_barriers(full);
    grid_launch_next();
    grid_wait();
    if (r.wq || r.wk) stage_weights<D>(r, s_w);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Me me;
    me.place(r, lane);
    auto rows = [&](int t, int j, int, uint32_t& bytes) {
        const Chunk c = chunk_of(r, j);
        bytes = c.n * D * 2;
        const __nv_bfloat16* p = c.what == 0 ? a.q + t * a.q_stride : c.what == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
        return reinterpret_cast<const uint8_t*>(p + c.h0 * D);
    };
    auto off = [&](int t, int j) {
        const Chunk c = chunk_of(r, j);
        if (c.what == 0) clear_rows<D>(r, c, a.q_out + t * a.q_out_stride);
    };
    feed<D, kBytes, 1, kRingPut, kWarpsPut>(r, dsmem + warp * Feed<D, kBytes, 1, kRingPut>::kWarp, full[warp], a.slots, rows, off,
                              [&](const Unit& u, const uint8_t* in, const float* table) {
        const Chunk c = chunk_of(r, u.j);
        if (c.what == 0) {
            __nv_bfloat16* to = a.q_out + u.t * a.q_out_stride;
            turn_rows<D, kWhole>(r, me, c, in, table, s_w, [&](int h) { return to + h * D; });
            return;
        }
        if (u.slot < 0 || u.slot >= a.num_slots) return;
        // Row of the cache that this token's head 0 is; head h is h pages of rows behind.
        const long long cell = (((long long)(u.slot >> a.ps_log2) * r.Hkv) << a.ps_log2) + (u.slot & ((1 << a.ps_log2) - 1));
        if constexpr (kFour) {
            put_rows<D, kWhole>(r, a, c, in, table, s_w, cell);
        } else if (c.what == 1) {
            __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(a.kp);
            turn_rows<D, kWhole>(r, me, c, in, table, s_w, [&](int h) { return to + (cell + ((long long)h << a.ps_log2)) * D; });
        } else {
            uint4* to = reinterpret_cast<uint4*>(a.vp);
            for (int i = lane; i < c.n * (D / 8); i += 32)
                to[(cell + ((long long)(c.h0 + i / (D / 8)) << a.ps_log2)) * (D / 8) + i % (D / 8)] = load16(in + i * 16);
        }
    });
}

// ---------------------------------------------------------------------- host

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// Whether n rows of `pb` bytes, `ps` apart, share a byte with n rows of `qb`
// bytes, `qs` apart.  Rows of different strides whose ranges meet count as sharing.
bool rows_meet(const void* p, size_t pb, size_t ps, const void* q, size_t qb, size_t qs, long long n) {
    if (!pb || !qb || n < 1) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    if (!(x < y + (n - 1) * qs + qb && y < x + (n - 1) * ps + pb)) return false;
    if (n == 1 || ps != qs) return true;
    const size_t off = y >= x ? (y - x) % ps : (ps - (x - y) % ps) % ps;   // q's rows behind p's, within a stride
    return off < pb || off + qb > ps;
}

// A strided operand of T tokens.
struct Rows {
    const void* p;
    size_t bytes, stride;    // of a token's row, between tokens
};
bool meet(const Rows& a, const Rows& b, long long T) { return rows_meet(a.p, a.bytes, a.stride, b.p, b.bytes, b.stride, T); }
// An output may be its input's own rows.
bool same(const Rows& a, const Rows& b, long long T) { return a.p == b.p && a.bytes == b.bytes && (a.stride == b.stride || T == 1); }
bool meet(const Span& s, const Rows& a, long long T) { return a.bytes && T > 0 && overlap_rows(s, a.p, T, a.bytes, a.stride); }

// What the rotation's own arguments have to be.  Without positions the tables have a row
// for every index that the T tokens take.
int check_rope(const float* cos, const float* sin, int max_pos, int rot, int d, int T, const int* positions, int seq_len, const void* wq,
               const void* wk, float eps) {
    if (!cos || !sin || max_pos < 1 || rot < 1 || rot > d) return FA_ERR_INVALID;
    if (!positions && (seq_len < 1 || (seq_len < T ? seq_len : T) > max_pos)) return FA_ERR_INVALID;
    if ((wq || wk) && !(eps >= 0.f && isfinite(eps))) return FA_ERR_INVALID;
    if (rot % 16) return FA_ERR_UNSUPPORTED;
    if (misaligned(cos, 15) || misaligned(sin, 15) || misaligned(positions, 3) || misaligned(wq, 15) || misaligned(wk, 15)) return FA_ERR_ALIGN;
    return FA_OK;
}
int check_heads(int T, int Hq, int Hkv, int d) {
    if (T < 0 || Hq < 0 || Hkv < 0 || Hq + (long long)Hkv < 1 || d < 1) return FA_ERR_INVALID;
    if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
    if ((long long)Hq * d > 0x3fffffff || (long long)Hkv * d > 0x3fffffff) return FA_ERR_UNSUPPORTED;
    // Units of one pass at the least: their number, and a step past it, fits 32 bits.
    const int pass = 512 / d;
    if (((Hq + pass - 1) / pass + 2LL * ((Hkv + pass - 1) / pass)) * T > 0x3fffffff) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// Blocks of `warps`, up to one an SM (the rings fill its shared memory).
int grid_for(int units, int sms, int warps) { return units < warps * sms ? (units + warps - 1) / warps : sms; }
// The rotation's arguments, with `arrays` of Hkv rows.  Rows a unit: as many as fill
// a slot, but no more than leave every warp a unit (whole passes).
RopeArgs rope_args(const float* cos, const float* sin, const int* positions, const void* wq, const void* wk, int T, int Hq, int Hkv, int max_pos, int rot,
                   int flags, int seq_len, int w_bf16, float eps, int pass, int most, int arrays, int workers, DevStatus* status) {
    int chunk = most, per_q, per_k;
    for (;; chunk /= 2) {
        per_q = (Hq + chunk - 1) / chunk;
        per_k = (Hkv + chunk - 1) / chunk;
        if (chunk == pass || (long long)T * (per_q + arrays * per_k) >= workers) break;
    }
    const int per = per_q + arrays * per_k;
    return {cos, sin, positions, wq, wk, T, Hq, Hkv, max_pos, rot, (flags & 0xff) != 0, seq_len, w_bf16 != 0, eps, chunk, per_q, per_k, per, T * per,
            (flags & FA_ROPE_CLEAR_Q ? 1 : 0) | (flags & FA_ROPE_CLEAR_K ? 2 : 0), status};
}
// Launches with `smem` bytes of dynamic shared memory, which a kernel is allowed once a device.
template <typename A>
int launch_rope(void (*kern)(RopeArgs, A), std::atomic<uint64_t>& prepared, int grid, int threads, uint32_t smem, cudaStream_t stream, const RopeArgs& r, const A& a) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_LAUNCH;
    if (!(prepared.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return FA_ERR_LAUNCH;
        prepared.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_dependent(kern, grid, threads, smem, stream, r, a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_qk_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, void* q_out, void* k_out, int64_t q_out_stride,
               int64_t k_out_stride, int T, int Hq, int Hkv, int d, const float* cos, const float* sin, int max_pos, int rot,
               int flags, const int* positions, int seq_len, const void* q_weight, const void* k_weight, int weights_bf16,
               float eps, cudaStream_t stream) {
    int rc = check_heads(T, Hq, Hkv, d);
    if (rc != FA_OK) return rc;
    if (T > 0 && ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)))) return FA_ERR_INVALID;
    rc = check_rope(cos, sin, max_pos, rot, d, T, positions, seq_len, q_weight, k_weight, eps);
    if (rc != FA_OK) return rc;
    const long long nq = (long long)Hq * d, nk = (long long)Hkv * d;
    if (Hq == 0) q = q_out = nullptr, q_stride = q_out_stride = 0;
    if (Hkv == 0) k = k_out = nullptr, k_stride = k_out_stride = 0;
    if (q_stride < nq || k_stride < nk || q_out_stride < nq || k_out_stride < nk) return FA_ERR_INVALID;
    if (misaligned(q, 15) || misaligned(k, 15) || misaligned(q_out, 15) || misaligned(k_out, 15) || (q_stride & 7) || (k_stride & 7) ||
        (q_out_stride & 7) || (k_out_stride & 7))
        return FA_ERR_ALIGN;
    if (T == 0) return FA_OK;
    const size_t w = weights_bf16 ? 2 : 4;
    const Rows in[] = {{q, (size_t)nq * 2, (size_t)q_stride * 2}, {k, (size_t)nk * 2, (size_t)k_stride * 2}};
    const Rows out[] = {{q_out, (size_t)nq * 2, (size_t)q_out_stride * 2}, {k_out, (size_t)nk * 2, (size_t)k_out_stride * 2}};
    const size_t table = (size_t)max_pos * rot * 2;
    const Span small[] = {{cos, table}, {sin, table}, {positions, positions ? 4 * (size_t)T : 0}, {q_weight, q_weight ? w * d : 0},
                          {k_weight, k_weight ? w * d : 0}};
    if (meet(out[0], out[1], T)) return FA_ERR_INVALID;
    for (int i = 0; i < 2; ++i) {
        for (const Span& s : small)
            if (meet(s, out[i], T)) return FA_ERR_INVALID;
        if (meet(out[i], in[1 - i], T) || (meet(out[i], in[i], T) && !same(out[i], in[i], T))) return FA_ERR_INVALID;
    }
    const int sms = fa_num_sms();
    DevStatus* status = device_status_ptr();
    if (sms < 1 || !status) return FA_ERR_LAUNCH;
    const RowsArgs a = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(q_out),
                        static_cast<__nv_bfloat16*>(k_out), q_stride, k_stride, q_out_stride, k_out_stride};
    auto launch = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        static std::atomic<uint64_t> prepared{0};
        const RopeArgs r = rope_args(cos, sin, positions, q_weight, k_weight, T, Hq, Hkv, max_pos, rot, flags, seq_len, weights_bf16, eps, kPass<D>, kChunk<D>, 1, kWarps * sms, status);
        return launch_rope(qk_rope_kernel<D>, prepared, grid_for(r.units, sms, kWarps), 32 * kWarps, kSmem<D>, stream, r, a);
    };
    if (d == 64) return launch(std::integral_constant<int, 64>{});
    if (d == 128) return launch(std::integral_constant<int, 128>{});
    return launch(std::integral_constant<int, 256>{});
}

size_t fa_qk_rope_bwd_workspace_size(int d) {
    if (d != 64 && d != 128 && d != 256) return 0;
    const int sms = fa_num_sms();
    return (size_t)(sms > 0 ? sms : kMaxSMs) * 2 * d * 4;      // a block an SM
}

int fa_qk_rope_bwd(const void* dq_out, const void* dk_out, int64_t dq_out_stride, int64_t dk_out_stride, const void* q, const void* k,
                   int64_t q_stride, int64_t k_stride, void* dq, void* dk, float* dq_weight, float* dk_weight, int T, int Hq, int Hkv,
                   int d, const float* cos, const float* sin, int max_pos, int rot, int flags, const int* positions, int seq_len,
                   const void* q_weight, const void* k_weight, int weights_bf16, float eps, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream) {
    int rc = check_heads(T, Hq, Hkv, d);
    if (rc != FA_OK) return rc;
    if (T > 0 && ((Hq > 0 && (!dq_out || !dq || (q_weight && !q))) || (Hkv > 0 && (!dk_out || !dk || (k_weight && !k))))) return FA_ERR_INVALID;
    if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr)) return FA_ERR_INVALID;
    rc = check_rope(cos, sin, max_pos, rot, d, T, positions, seq_len, q_weight, k_weight, eps);
    if (rc != FA_OK) return rc;
    const long long nq = (long long)Hq * d, nk = (long long)Hkv * d;
    if (Hq == 0) dq_out = q = dq = nullptr, dq_out_stride = q_stride = 0;
    if (Hkv == 0) dk_out = k = dk = nullptr, dk_out_stride = k_stride = 0;
    if (dq_out_stride < nq || dk_out_stride < nk || (q_weight && q_stride < nq) || (k_weight && k_stride < nk)) return FA_ERR_INVALID;
    if (misaligned(dq_out, 15) || misaligned(dk_out, 15) || misaligned(dq, 15) || misaligned(dk, 15) || (q_weight && (misaligned(q, 15) || (q_stride & 7))) ||
        (k_weight && (misaligned(k, 15) || (k_stride & 7))) || misaligned(dq_weight, 15) || misaligned(dk_weight, 15) || (dq_out_stride & 7) || (dk_out_stride & 7))
        return FA_ERR_ALIGN;
    const bool norm = q_weight || k_weight;
    if (norm && (!workspace || misaligned(workspace, 255) || workspace_bytes < fa_qk_rope_bwd_workspace_size(d))) return FA_ERR_WORKSPACE;
    const size_t w = weights_bf16 ? 2 : 4, table = (size_t)max_pos * rot * 2;
    const Rows in[] = {{dq_out, (size_t)nq * 2, (size_t)dq_out_stride * 2},
                       {dk_out, (size_t)nk * 2, (size_t)dk_out_stride * 2},
                       {q, q_weight ? (size_t)nq * 2 : 0, (size_t)q_stride * 2},
                       {k, k_weight ? (size_t)nk * 2 : 0, (size_t)k_stride * 2}};
    const Rows out[] = {{dq, (size_t)nq * 2, (size_t)nq * 2}, {dk, (size_t)nk * 2, (size_t)nk * 2}};
    const Span small[] = {{cos, table}, {sin, table}, {positions, positions ? 4 * (size_t)T : 0}, {q_weight, q_weight ? w * d : 0},
                          {k_weight, k_weight ? w * d : 0}};
    const Span sums[] = {{dq_weight, dq_weight ? 4 * (size_t)d : 0}, {dk_weight, dk_weight ? 4 * (size_t)d : 0},
                         {workspace, norm ? fa_qk_rope_bwd_workspace_size(d) : 0}};
    if (meet(out[0], out[1], T)) return FA_ERR_INVALID;
    for (int i = 0; i < 2; ++i) {
        for (const Span& s : small)
            if (meet(s, out[i], T)) return FA_ERR_INVALID;
        for (const Span& s : sums)
            if (meet(s, out[i], T)) return FA_ERR_INVALID;
        // A gradient may take the place of the rows that it is computed from, one for one.
        for (int j = 0; j < 4; ++j)
            if (meet(out[i], in[j], T) && !((j & 1) == i && same(out[i], in[j], T))) return FA_ERR_INVALID;
    }
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(sums[i], sums[j])) return FA_ERR_INVALID;
        for (const Span& s : small)
            if (overlap(sums[i], s)) return FA_ERR_INVALID;
        for (const Rows& x : in)
            if (meet(sums[i], x, T)) return FA_ERR_INVALID;
    }
    if (T == 0 && !norm) return FA_OK;
    const int sms = fa_num_sms();
    DevStatus* status = device_status_ptr();
    if (sms < 1 || !status) return FA_ERR_LAUNCH;
    const GradArgs a = {static_cast<const __nv_bfloat16*>(dq_out), static_cast<const __nv_bfloat16*>(dk_out), static_cast<const __nv_bfloat16*>(q),
                        static_cast<const __nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk),
                        dq_out_stride, dk_out_stride, q_stride, k_stride, static_cast<float*>(workspace)};
    int grid = 0;
    auto launch = [&](auto dim) -> int {
        constexpr int D = decltype(dim)::value;
        static std::atomic<uint64_t> prepared{0};
        const RopeArgs r = rope_args(cos, sin, positions, q_weight, k_weight, T, Hq, Hkv, max_pos, rot, flags, seq_len, weights_bf16, eps, kPass<D>, kChunkGrad<D>, 1, kWarpsGrad * sms, status);
        grid = grid_for(r.units, sms, kWarpsGrad);
        return grid < 1 ? FA_OK : launch_rope(qk_rope_bwd_kernel<D>, prepared, grid, 32 * kWarpsGrad, kSmemGrad<D>, stream, r, a);
    };
    rc = d == 64 ? launch(std::integral_constant<int, 64>{}) : d == 128 ? launch(std::integral_constant<int, 128>{}) : launch(std::integral_constant<int, 256>{});
    if (rc != FA_OK || !norm) return rc;
    return launch_dependent(qk_rope_dw_kernel, 2 * d / 32, 1024, 0, stream, a.partial, grid, d, dq_weight, dk_weight) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_rope_store(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out,
                  int64_t q_out_stride, int T, int Hq, int Hkv, int d, const float* cos, const float* sin, int max_pos, int rot,
                  int flags, const int* positions, const void* q_weight, const void* k_weight, int weights_bf16, float eps,
                  const int* slots, void* k_pages, void* v_pages, void* k_scales, void* v_scales, int num_pages, int page_size,
                  cudaStream_t stream) {
    int rc = check_heads(T, Hq, Hkv, d);
    if (rc != FA_OK) return rc;
    if (!k || !v || !slots || !positions || !k_pages || !v_pages || Hkv < 1 || num_pages < 1) return FA_ERR_INVALID;
    if ((Hq > 0 && (!q || !q_out)) || (k_scales != nullptr) != (v_scales != nullptr)) return FA_ERR_INVALID;
    rc = check_rope(cos, sin, max_pos, rot, d, T, positions, 1, q_weight, k_weight, eps);
    if (rc != FA_OK) return rc;
    const int lg = page_log2(page_size);
    if (lg < 0 || (long long)num_pages * page_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    const long long nq = (long long)Hq * d, nk = (long long)Hkv * d;
    if (Hq == 0) q = q_out = nullptr, q_stride = q_out_stride = 0;
    if (q_stride < nq || k_stride < nk || v_stride < nk || q_out_stride < nq) return FA_ERR_INVALID;
    if (misaligned(q, 15) || misaligned(k, 15) || misaligned(v, 15) || misaligned(q_out, 15) || (q_stride & 7) || (k_stride & 7) ||
        (v_stride & 7) || (q_out_stride & 7) || misaligned(k_pages, 15) || misaligned(v_pages, 15) || misaligned(k_scales, 15) ||
        misaligned(v_scales, 15) || misaligned(slots, 3))
        return FA_ERR_ALIGN;
    if (T == 0) return FA_OK;
    const bool four = k_scales != nullptr;
    const size_t w = weights_bf16 ? 2 : 4, table = (size_t)max_pos * rot * 2, cells = (size_t)num_pages * page_size * Hkv;
    const size_t pages = cells * (four ? d / 2 : 2 * d), scales = four ? cells * (d / 32) : 0;
    const Rows in[] = {{q, (size_t)nq * 2, (size_t)q_stride * 2}, {k, (size_t)nk * 2, (size_t)k_stride * 2}, {v, (size_t)nk * 2, (size_t)v_stride * 2}};
    const Rows out = {q_out, (size_t)nq * 2, (size_t)q_out_stride * 2};
    const Span small[] = {{cos, table}, {sin, table}, {positions, 4 * (size_t)T}, {slots, 4 * (size_t)T}, {q_weight, q_weight ? w * d : 0},
                          {k_weight, k_weight ? w * d : 0}};
    const Span cache[] = {{k_pages, pages}, {v_pages, pages}, {k_scales, scales}, {v_scales, scales}};
    if ((meet(out, in[0], T) && !same(out, in[0], T)) || meet(out, in[1], T) || meet(out, in[2], T)) return FA_ERR_INVALID;
    for (const Span& s : small)
        if (meet(s, out, T)) return FA_ERR_INVALID;
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(cache[i], cache[j])) return FA_ERR_INVALID;
        for (const Span& s : small)
            if (overlap(cache[i], s)) return FA_ERR_INVALID;
        for (const Rows& x : in)
            if (meet(cache[i], x, T)) return FA_ERR_INVALID;
        if (meet(cache[i], out, T)) return FA_ERR_INVALID;
    }
    const int sms = fa_num_sms();
    DevStatus* status = device_status_ptr();
    if (sms < 1 || !status) return FA_ERR_LAUNCH;
    const PutArgs a = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                       static_cast<__nv_bfloat16*>(q_out), q_stride, k_stride, v_stride, q_out_stride, slots, static_cast<uint8_t*>(k_pages),
                       static_cast<uint8_t*>(v_pages), static_cast<uint8_t*>(k_scales), static_cast<uint8_t*>(v_scales), lg,
                       (long long)num_pages * page_size};
    auto launch = [&](auto dim, auto bits4) {
        constexpr int D = decltype(dim)::value;
        constexpr bool kFour = decltype(bits4)::value;
        static std::atomic<uint64_t> prepared[2];
        const bool whole = rot == D && !(flags & 0xff);
        const RopeArgs r = rope_args(cos, sin, positions, q_weight, k_weight, T, Hq, Hkv, max_pos, rot, flags, 1, weights_bf16, eps, kPass<D>, kChunk<D>, 2, kWarpsPut * sms, status);
        return launch_rope(whole ? rope_store_kernel<D, kFour, true> : rope_store_kernel<D, kFour, false>, prepared[whole], grid_for(r.units, sms, kWarpsPut), 32 * kWarpsPut, kSmemPut<D>, stream, r, a);
    };
    auto pick = [&](auto bits4) {
        return d == 64 ? launch(std::integral_constant<int, 64>{}, bits4) : d == 128 ? launch(std::integral_constant<int, 128>{}, bits4)
                                                                                 : launch(std::integral_constant<int, 256>{}, bits4);
    };
    return four ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // extern "C"

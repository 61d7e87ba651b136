// fa_prefix.cu -- fa_prefix_fwd: attention of new tokens over a shared prefix
// and each request's own paged keys.
#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"
#include "fa_internal.h"

namespace fa {
namespace {

struct PrefixArgs {
    const __nv_bfloat16 *q, *kp, *vp;
    __nv_bfloat16* o;
    float* lse;
    const int *table, *kv_lens, *cu, *prefix_table;
    DevStatus* status;
    long long q_stride;
    int T, B, Hq, Hkv, W, P, ps_log2, prefix_len, max_seqlen;
    float scale_log2;
};

// One warp a (token, head); lane l holds elements l, l + 32, ... of the row.
template <int D>
__global__ void __launch_bounds__(256) prefix_simple_kernel(const PrefixArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = blockIdx.x * 8LL + (threadIdx.x >> 5);
    if (w >= (long long)a.T * a.Hq) return;
    const int t = (int)(w / a.Hq), h = (int)(w % a.Hq), hk = h / (a.Hq / a.Hkv);
    int b = -1, c0 = 0, c1 = 0, prev = 0;
    for (int i = 0; i <= a.B; ++i) {   // sanitised offsets
        int c = a.cu ? a.cu[i] : i;
        c = c < 0 ? 0 : (c > a.T ? a.T : c);
        c = c > prev ? c : prev;
        if (i > 0 && c - prev > a.max_seqlen) {
            if (lane == 0) atomicCAS(&a.status->code, 0, -1);
            return;
        }
        if (i > 0 && b < 0 && t >= prev && t < c) { b = i - 1; c0 = prev; c1 = c; }
        prev = c;
    }
    if (b < 0) return;
    const int cap = a.W << a.ps_log2, ps = 1 << a.ps_log2;
    int s = a.kv_lens[b];
    s = s < 0 ? 0 : (s > cap ? cap : s);
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) { q[e] = __bfloat162float(a.q[t * a.q_stride + h * D + e * 32 + lane]); o[e] = 0.f; }
    for (int part = 0; part < 2; ++part) {
        const int* tab = part ? a.table + (long long)b * a.W : a.prefix_table;
        const int n = part ? s - (c1 - c0) + (t - c0) + 1 : a.prefix_len;
        for (int j = 0; j < n; ++j) {
            const int page = tab[j >> a.ps_log2];
            if (page < 0 || page >= a.P) continue;
            const long long row = ((((long long)page * a.Hkv + hk) << a.ps_log2) + (j & (ps - 1))) * D + lane;
            float x = 0.f;
            for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(a.kp[row + e * 32]);
            for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
            x *= a.scale_log2;
            const float mn = fmaxf(m, x);
            const float f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(x - mn);
            l = l * f + p;
            for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * __bfloat162float(a.vp[row + e * 32]);
            m = mn;
        }
    }
    for (int e = 0; e < E; ++e)
        a.o[((long long)t * a.Hq + h) * D + e * 32 + lane] = __float2bfloat16(l > 0.f ? o[e] / l : 0.f);
    if (lane == 0) a.lse[(long long)h * a.T + t] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_prefix_workspace_size(int T, int B, int Hq, int Hkv, int d, int max_seqlen) {
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 128 || max_seqlen < 1 ||
        (d != 64 && d != 128 && d != 256))
        return 0;
    return 256;
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
    const size_t need = fa_prefix_workspace_size(T, B, Hq, Hkv, d, max_seqlen);
    if (!workspace || misaligned(workspace, 255) || workspace_bytes < need) return FA_ERR_WORKSPACE;
    DevStatus* status = device_status_ptr();
    if (!status) return FA_ERR_LAUNCH;
    PrefixArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.kp = static_cast<const __nv_bfloat16*>(k_pages);
    a.vp = static_cast<const __nv_bfloat16*>(v_pages);
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.table = block_table;
    a.kv_lens = kv_lens;
    a.cu = cu_seqlens;
    a.prefix_table = prefix_table;
    a.status = status;
    a.q_stride = q_stride;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.W = table_width;
    a.P = num_pages;
    a.ps_log2 = lg;
    a.prefix_len = prefix_len;
    a.max_seqlen = max_seqlen;
    a.scale_log2 = alpha * 1.4426950408889634f;
    const int grid = (int)(((long long)T * Hq + 7) / 8);
    if (d == 64) prefix_simple_kernel<64><<<grid, 256, 0, stream>>>(a);
    else if (d == 128) prefix_simple_kernel<128><<<grid, 256, 0, stream>>>(a);
    else prefix_simple_kernel<256><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

}  // extern "C"

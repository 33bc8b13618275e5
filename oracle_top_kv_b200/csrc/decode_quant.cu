// decode_quant.cu -- decode step of the full layer over a quantised cache: it
// attends to every cached row and selects the index set of the new token, as
// decode_full.cu does over a bf16 cache, with other kernels:
//
//  1. decode_quant_full_kernel: the caches' steps (32 4-bit or 16 8-bit keys
//     each) of all (sequence, KV group) units, laid end to end, are cut into
//     equal shares, one per CTA of a grid that fills the GPU once: ragged
//     batches and few long sequences keep every SM busy alike.  A CTA writes
//     one partial (m, l, O) per unit that its share touches.
//  2. decode_quant_combine_kernel: exact log-sum-exp merge -> o, lse, lse2.
//  3. decode_quant_select_kernel: the group score max_h (a2_h - lse2_h) needs
//     every head's final lse.  Instead of carrying every logit from pass 1
//     (64 bytes written and read per key against rows of 68 or 132) it reads the K rows
//     again and recomputes the logits of its slice straight into shared memory,
//     where the slice's top-(k - w) is found.  Its merge is decode_full.cu's.
//  k - w > 1024: decode_quant_select_one_kernel, one CTA per unit.
//  sel_scores: decode_quant_sel_scores_kernel rescores the selected keys.
#include <atomic>

#include "block_topk.cuh"
#include "cta_select.cuh"
#include "hs_common.cuh"
#include "hs_kernels.cuh"
#include "quant_kv.cuh"

namespace hs {
namespace dq {

constexpr int kWarps = 4;
constexpr int kMaxCtas = 640;  // partial slots reserved: at most kMaxCtas + units
template <int F> constexpr int kStep = F == HS_KV_INT4 ? 32 : 16;

struct Ws {
    float* part;   // [kMaxCtas + units][kPart]
    float* lse2;   // [batch * hq]
    uint64_t* cand;
    int* cand_n;
    uint64_t* cand2;
    int* cand2_n;
    int n_sel, n_grp;
    size_t bytes;
};

static Ws ws_layout(const KParams& p, void* base) {
    Ws w;
    const size_t units = (size_t)p.batch * p.hkv;
    w.n_sel = sel_splits(p);
    w.n_grp = sel_groups(w.n_sel);
    char* c = static_cast<char*>(base);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* r = c + at;
        at += align256(bytes);
        return r;
    };
    w.part = (float*)take((kMaxCtas + units) * (32 + 16 * p.head_dim) * sizeof(float));
    w.lse2 = (float*)take((size_t)p.batch * p.hq * sizeof(float));
    w.cand = (uint64_t*)take(units * w.n_sel * kSelMaxRanked * sizeof(uint64_t));
    w.cand_n = (int*)take(units * w.n_sel * sizeof(int));
    w.cand2 = (uint64_t*)take(units * w.n_grp * kSelMaxRanked * sizeof(uint64_t));
    w.cand2_n = (int*)take(units * w.n_grp * sizeof(int));
    w.bytes = at;
    return w;
}

// Steps of sequence b's cache (per unit); none for a length out of range.
template <int NK>
__device__ __forceinline__ int seq_steps(const int32_t* seq_len, int b, int t_kv) {
    const int L = __ldg(seq_len + b);
    return L >= 1 && L <= t_kv ? (L + NK - 1) / NK : 0;
}

// Sum over sequences b0 <= b < b1 of their steps, by one warp (all lanes get it).
template <int NK>
__device__ __forceinline__ long long sum_steps(const int32_t* seq_len, int b0, int b1, int t_kv) {
    long long s = 0;
    for (int b = b0 + (threadIdx.x & 31); b < b1; b += 32) s += seq_steps<NK>(seq_len, b, t_kv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// CTAs of a grid of G that get a share of `total` steps: at least a step per
// warp each, so that none between two others is empty.
__device__ __forceinline__ int ctas_used(int G, long long total) {
    return (int)min((long long)G, max(1ll, total / kWarps));
}
// CTA c of G used ones takes steps [share(c), share(c + 1)) of `total`.
__device__ __forceinline__ long long share(int c, int G, long long total) { return total * c / G; }
// The CTA whose share holds step x.
__device__ __forceinline__ int share_of(long long x, int G, long long total) {
    return (int)(((x + 1) * G - 1) / total);
}

template <int D, int F>
__global__ void __launch_bounds__(kWarps * 32)
    decode_quant_full_kernel(KParams p, QuantCache cache, const __nv_bfloat16* __restrict__ q,
                             const int32_t* __restrict__ seq_len, float* __restrict__ part) {
    constexpr int NK = kStep<F>;
    using A = QAttend<D, F, NK>;
    extern __shared__ __align__(16) float smem[];  // kWarps partials
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = p.group;
    const long long total = sum_steps<NK>(seq_len, 0, p.batch, p.t_kv) * p.hkv;
    const int G = ctas_used(gridDim.x, total);
    if (total == 0 || (int)blockIdx.x >= G) return;
    long long at = share(blockIdx.x, G, total);
    const long long end = share(blockIdx.x + 1, G, total);
    // the sequence that holds step `at`: 32 at a time
    int b = 0;
    long long before = 0;  // steps of the units before sequence b
    for (;; b += 32) {
        const long long mine =
            b + lane < p.batch ? (long long)seq_steps<NK>(seq_len, b + lane, p.t_kv) * p.hkv : 0;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + incl > at);
        if (past) {
            const int x = __ffs(past) - 1;
            before += __shfl_sync(0xffffffffu, incl - mine, x);
            b += x;
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    int n = seq_steps<NK>(seq_len, b, p.t_kv);
    int u = (int)((at - before) / n);
    int s0 = (int)((at - before) - (long long)u * n);
    while (at < end) {
        const int s1 = (int)min((long long)n, s0 + (end - at));
        const int unit = b * p.hkv + u;
        A st;
        st.init(q + ((size_t)b * p.hq + (size_t)u * g) * D, D, g);
        const QuantCache uc = unit_cache<D, F>(p, cache, unit);
        const int L = __ldg(seq_len + b);
        if (p.bt) st.run(uc, QPagedRange{0, L, page_map(p, b, u)}, s0 + warp, kWarps, s1, p.scale_log2);
        else st.run(uc, QRange{0, L}, s0 + warp, kWarps, s1, p.scale_log2);
        st.finish();
        st.store_part(smem + warp * A::kPart, g);
        __syncthreads();
        float* dst = part + (size_t)(blockIdx.x + unit) * A::kPart;
        for (int e = threadIdx.x; e < g * (D / 4); e += blockDim.x) {
            const int h = e / (D / 4);
            float M = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, smem[w * A::kPart + 2 * h]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* pw = smem + w * A::kPart;
                const float f = sq::merge_weight(pw[2 * h], M);
                const float4 x = reinterpret_cast<const float4*>(pw + 32)[e];
                l += pw[2 * h + 1] * f;
                acc.x += x.x * f;
                acc.y += x.y * f;
                acc.z += x.z * f;
                acc.w += x.w * f;
            }
            reinterpret_cast<float4*>(dst + 32)[e] = acc;
            if (e % (D / 4) == 0) {
                dst[2 * h] = M;
                dst[2 * h + 1] = l;
            }
        }
        __syncthreads();  // the partials are read before the next unit's
        at += s1 - s0;
        s0 = 0;
        if (++u == p.hkv) {
            u = 0;
            do { ++b; } while (b < p.batch && (n = seq_steps<NK>(seq_len, b, p.t_kv)) == 0);
        }
    }
}

// One CTA per (sequence, head), `parts` x D threads: thread (part, d) adds up
// element d of every parts-th partial of the unit.
constexpr int kParts = 4;
template <int D, int F>
__global__ void __launch_bounds__(kParts * D)
    decode_quant_combine_kernel(KParams p, const float* __restrict__ part, int grid,
                                const int32_t* __restrict__ seq_len,
                                __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                                float* __restrict__ lse2) {
    constexpr int NK = kStep<F>, kPart = 32 + 16 * D;
    __shared__ float s_acc[kParts][D], s_m[kParts * D / 32], s_l[kParts * D / 32];
    const int row = blockIdx.x, h = row % p.hq, b = row / p.hq;
    const int u = h / p.group, hh = h % p.group, unit = b * p.hkv + u;
    const int tid = threadIdx.x, warp = tid >> 5, d = tid % D, prt = tid / D;
    const int n = seq_steps<NK>(seq_len, b, p.t_kv);
    if (n == 0) {  // length out of range
        if (tid < D) o[(size_t)row * D + d] = __float2bfloat16_rn(0.f);
        if (tid == 0) {
            lse[row] = lse2[row] = -INFINITY;
            set_status(HS_ERR_BOUNDS);
        }
        return;
    }
    const long long before = sum_steps<NK>(seq_len, 0, b, p.t_kv);
    const long long total = (before + sum_steps<NK>(seq_len, b, p.batch, p.t_kv)) * p.hkv;
    const long long first = before * p.hkv + (long long)u * n;
    const int G = ctas_used(grid, total);
    const int c0 = share_of(first, G, total), c1 = share_of(first + n - 1, G, total);
    const float* base = part + (size_t)(c0 + unit) * kPart;
    const int cnt = c1 - c0 + 1;
    float M = -INFINITY;
    for (int c = tid; c < cnt; c += kParts * D) M = fmaxf(M, base[(size_t)c * kPart + 2 * hh]);
    M = warp_max(M);
    if ((tid & 31) == 0) s_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kParts * D / 32; ++w) M = fmaxf(M, s_m[w]);
    float l = 0.f, acc = 0.f;
    for (int c = tid; c < cnt; c += kParts * D) {
        const float* pc = base + (size_t)c * kPart;
        l += pc[2 * hh + 1] * sq::merge_weight(pc[2 * hh], M);
    }
    l = warp_sum(l);
    if ((tid & 31) == 0) s_l[warp] = l;
#pragma unroll 4
    for (int c = prt; c < cnt; c += kParts) {
        const float* pc = base + (size_t)c * kPart;
        acc += pc[32 + hh * D + d] * sq::merge_weight(pc[2 * hh], M);
    }
    s_acc[prt][d] = acc;
    __syncthreads();
    if (prt != 0) return;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kParts * D / 32; ++w) l += s_l[w];
#pragma unroll
    for (int x = 1; x < kParts; ++x) acc += s_acc[x][d];
    o[(size_t)row * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
    if (d == 0) {
        const float l2 = l == 0.f ? -INFINITY : M + log2f(l);
        lse[row] = l2 * kLn2;
        lse2[row] = l2;
    }
}

// -------------------------------------------------------------- group scores
// Group scores of 16 keys by one warp, log2 domain: the keys are the 16 rows
// (A) and the heads the columns (B), so a key's heads lie in one quad.
template <int D, int F>
struct QScore {
    using R = QRow<D, F>;
    uint32_t qb[2][D / 16][2];  // B fragments, heads 0..7 and 8..15
    float qs[2][2], nl[2][2];   // heads 8 n + 2 t + e: scale_log2 sum(q), -lse2
    float scale_log2;

    __device__ __forceinline__ void init(const __nv_bfloat16* q, const float* lse2, int g,
                                         float scale) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
        scale_log2 = scale;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int h = 8 * n + gid;
            __nv_bfloat16 x[D / 4];
            const uint4* src = reinterpret_cast<const uint4*>(q + (size_t)h * D + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                reinterpret_cast<uint4*>(x)[i] = h < g ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) sum += __bfloat162float(x[i]);
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __nv_bfloat162 pr =
                        __halves2bfloat162(x[k_dim<F>(ks, 2 * e)], x[k_dim<F>(ks, 2 * e + 1)]);
                    qb[n][ks][e] = *reinterpret_cast<const uint32_t*>(&pr);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hc = 8 * n + 2 * t + e;
                qs[n][e] = __shfl_sync(0xffffffffu, sum, (2 * t + e) * 4) * scale;
                nl[n][e] = hc < g ? -lse2[hc] : -INFINITY;
            }
        }
    }
    struct Regs {
        uint32_t k[2][R::kKW], e[2];
    };
    // rows of keys gid and gid + 8 (-1: none)
    __device__ __forceinline__ static void load(Regs& r, const QuantCache& c, int r0, int r1) {
        const int t = threadIdx.x & 3;
        ldg_words<R::kKW>(r.k[0], c.kc + (size_t)r0 * R::kBytes + t * (R::kBytes / 4), r0 >= 0);
        ldg_words<R::kKW>(r.k[1], c.kc + (size_t)r1 * R::kBytes + t * (R::kBytes / 4), r1 >= 0);
        r.e[0] = r0 >= 0 ? __ldg(c.ks + r0) : 0u;
        r.e[1] = r1 >= 0 ? __ldg(c.ks + r1) : 0u;
    }
    // Scores of keys gid (.x) and gid + 8 (.y), the same in all lanes of a quad.
    __device__ __forceinline__ float2 score(const Regs& r) const {
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t a[4];
            k_frag<F>(r.k[0], ks, a[0], a[2]);
            k_frag<F>(r.k[1], ks, a[1], a[3]);
            mma_bf16(s[0], a, qb[0][ks][0], qb[0][ks][1]);
            mma_bf16(s[1], a, qb[1][ks][0], qb[1][ks][1]);
        }
        float best[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float sc = entry_scale(r.e[k]);
            float z = entry_zero(r.e[k]);
            if constexpr (F == HS_KV_INT4) z = fmaf(8.f, sc, z);
            const float s2 = sc * scale_log2;
            float v = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    v = fmaxf(v, fmaf(s[n][2 * k + e], s2, qs[n][e] * z) + nl[n][e]);
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            best[k] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        }
        return make_float2(best[0], best[1]);
    }
};

// Row of logical key `key` of unit (b, u), relative to unit_cache's bases.
__device__ __forceinline__ int key_row(const KParams& p, const PageMap& pm, int key) {
    return p.bt ? pm.row(key) : key;
}

// Scores of keys first .. first + n - 1, by all warps of the CTA, to
// put(i, score) with i = 0 .. n - 1.
template <int D, int F, class Put>
__device__ __forceinline__ void score_keys(const QScore<D, F>& sc, const KParams& p,
                                           const QuantCache& c, const PageMap& pm, int first, int n,
                                           Put put) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    using S = QScore<D, F>;
    auto row = [&](int i) { return i < n ? key_row(p, pm, first + i) : -1; };
    typename S::Regs a, b;
    int i = warp * 16;
    if (i < n) S::load(a, c, row(i + gid), row(i + gid + 8));
    for (; i < n; i += nw * 16) {
        const int nx = i + nw * 16;
        if (nx < n) S::load(b, c, row(nx + gid), row(nx + gid + 8));
        const float2 v = sc.score(a);
        const int k = i + gid + 8 * t;
        if (t < 2 && k < n) put(k, t == 0 ? v.x : v.y);
        a = b;
    }
}

// Slice of the ranked keys 0..t-w of unit blockIdx.x / n_sel: its top-(k-w).
template <int D, int F>
__global__ void __launch_bounds__(kSelectThreads)
    decode_quant_select_kernel(KParams p, QuantCache cache, const __nv_bfloat16* __restrict__ q,
                               const int32_t* __restrict__ seq_len, Ws ws) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ CtaSelectSmem cs;
    __shared__ int s_n;
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem_raw);  // [kSelSlice]
    const int unit = blockIdx.x / ws.n_sel, sp = blockIdx.x % ws.n_sel;
    const int u = unit % p.hkv, b = unit / p.hkv;
    const int L = seq_len[b];
    const int Kc = p.k - p.window;
    int* out_n = ws.cand_n + (size_t)unit * ws.n_sel + sp;
    if (L < 1 || L > p.t_kv || L <= p.k || Kc <= 0) {  // nothing ranked here
        if (threadIdx.x == 0) *out_n = 0;
        return;
    }
    const int lo = L - p.window;  // ranked keys 0..lo-1
    const int per = (lo + ws.n_sel - 1) / ws.n_sel;  // <= kSelSlice
    const int i0 = sp * per;
    const int n = max(0, min(lo, i0 + per) - i0);
    const size_t head0 = (size_t)b * p.hq + (size_t)u * p.group;
    QScore<D, F> sc;
    sc.init(q + head0 * D, ws.lse2 + head0, p.group, p.scale_log2);
    score_keys<D, F>(sc, p, unit_cache<D, F>(p, cache, unit), page_map(p, b, u), i0, n,
                     [&](int i, float v) { bits[i] = float_order(v); });
    __syncthreads();
    auto key = [&](int i) -> uint64_t {
        return ((uint64_t)bits[i] << 32) | (uint64_t)(0xffffffffu - (uint32_t)(i0 + i));
    };
    uint64_t* dst = ws.cand + ((size_t)unit * ws.n_sel + sp) * kSelMaxRanked;
    if (n <= Kc) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = key(i);
        if (threadIdx.x == 0) *out_n = n;
        return;
    }
    const uint64_t kth = cta_kth_largest(key, n, Kc, cs);
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint64_t v = key(i);
        if (v >= kth) dst[atomicAdd(&s_n, 1)] = v;
    }
    __syncthreads();
    if (threadIdx.x == 0) *out_n = s_n;  // exactly Kc: the keys are distinct
}

// Budgets k - w above kSelMaxRanked: one CTA per unit streams the scores
// through an exact top-k buffer.
constexpr int kOneRound = kSelectThreads;  // keys offered per round
template <int D, int F>
__global__ void __launch_bounds__(kSelectThreads)
    decode_quant_select_one_kernel(KParams p, QuantCache cache,
                                   const __nv_bfloat16* __restrict__ q,
                                   const int32_t* __restrict__ seq_len, Ws ws,
                                   int32_t* __restrict__ idx, int32_t* __restrict__ cnt) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ int s_count;
    __shared__ unsigned long long s_thresh;
    __shared__ float s_score[kOneRound];
    const int unit = blockIdx.x, u = unit % p.hkv, b = unit / p.hkv;
    const int L = seq_len[b];
    int32_t* irow = idx + (size_t)unit * p.ksel;
    if (L < 1 || L > p.t_kv || L <= p.k) {  // no row, or the budget covers every key
        const int n = L < 1 || L > p.t_kv ? 0 : L;
        for (int x = threadIdx.x; x < p.ksel; x += blockDim.x) irow[x] = x < n ? x : -1;
        if (threadIdx.x == 0) cnt[unit] = n;
        return;
    }
    const int lo = L - p.window;
    BlockTopK topk;
    topk.setup(smem_raw, p.k - p.window, kOneRound, &s_count, &s_thresh);
    const size_t head0 = (size_t)b * p.hq + (size_t)u * p.group;
    QScore<D, F> sc;
    sc.init(q + head0 * D, ws.lse2 + head0, p.group, p.scale_log2);
    const QuantCache uc = unit_cache<D, F>(p, cache, unit);
    const PageMap pm = page_map(p, b, u);
    __syncthreads();
    for (int i0 = 0; i0 < lo; i0 += kOneRound) {
        const int n = min(kOneRound, lo - i0);
        score_keys<D, F>(sc, p, uc, pm, i0, n, [&](int i, float v) { s_score[i] = v; });
        __syncthreads();
        if ((int)threadIdx.x < n) topk.offer(s_score[threadIdx.x], (uint32_t)(i0 + threadIdx.x));
        topk.end_round();
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int n_out = topk.finish(irow, nullptr, p.ksel, lo, L - 1);
    if (threadIdx.x == 0) cnt[unit] = n_out;
}

// sel_scores: max_h p of every selected key.
template <int D, int F>
__global__ void __launch_bounds__(128)
    decode_quant_sel_scores_kernel(KParams p, QuantCache cache,
                                   const __nv_bfloat16* __restrict__ q, const float* lse2,
                                   const int32_t* __restrict__ idx,
                                   const int32_t* __restrict__ cnt, float* __restrict__ sel) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x, u = unit % p.hkv, b = unit / p.hkv;
    const size_t head0 = (size_t)b * p.hq + (size_t)u * p.group;
    const int n = cnt[unit];
    QScore<D, F> sc;
    sc.init(q + head0 * D, lse2 + head0, p.group, p.scale_log2);
    const QuantCache uc = unit_cache<D, F>(p, cache, unit);
    const PageMap pm = page_map(p, b, u);
    const int32_t* irow = idx + (size_t)unit * p.ksel;
    for (int i = 16 * (blockIdx.y * 4 + warp); i < p.ksel; i += 64 * gridDim.y) {
        int r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int x = i + gid + 8 * k;
            r[k] = x < n ? key_row(p, pm, irow[x]) : -1;
        }
        typename QScore<D, F>::Regs regs;
        QScore<D, F>::load(regs, uc, r[0], r[1]);
        const float2 v = sc.score(regs);
        const int x = i + gid + 8 * t;
        if (t < 2 && x < p.ksel)
            sel[(size_t)unit * p.ksel + x] = x < n ? exp2f(t == 0 ? v.x : v.y) : 0.f;
    }
}

// CTAs of the full kernel that fill the current device once (cached per device).
template <int D, int F>
static cudaError_t full_grid(size_t smem, int* ctas) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        int sms = 0, per = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return e;
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                 &per, decode_quant_full_kernel<D, F>, kWarps * 32, smem)) != cudaSuccess)
            return e;
        n = min(kMaxCtas, max(1, per) * sms);
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *ctas = n;
    return cudaSuccess;
}

template <int D, int F>
static cudaError_t launch_t(const KParams& p, const QuantCache& c, const void* q_,
                            const int32_t* seq_len, int32_t* idx, int32_t* cnt, void* o,
                            float* lse, float* sel, void* ws_, cudaStream_t st) {
    using A = QAttend<D, F, kStep<F>>;
    const __nv_bfloat16* q = (const __nv_bfloat16*)q_;
    const Ws w = ws_layout(p, ws_);
    const int units = p.batch * p.hkv;
    cudaError_t e;
    auto full = decode_quant_full_kernel<D, F>;
    const size_t smem = kWarps * A::kPart * sizeof(float);
    if ((e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
        cudaSuccess)
        return e;
    int G = 0;
    if ((e = full_grid<D, F>(smem, &G)) != cudaSuccess) return e;
    // no CTA below a step per warp, as far as the capacity tells
    const long long most = (long long)units * ((p.t_kv + kStep<F> - 1) / kStep<F>);
    G = (int)max(1ll, min((long long)G, (most + kWarps - 1) / kWarps));
    full<<<G, kWarps * 32, smem, st>>>(p, c, q, seq_len, w.part);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    decode_quant_combine_kernel<D, F><<<p.batch * p.hq, kParts * D, 0, st>>>(
        p, w.part, G, seq_len, (__nv_bfloat16*)o, lse, w.lse2);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int Kc = p.k - p.window;
    if (Kc <= kSelMaxRanked) {
        auto select = decode_quant_select_kernel<D, F>;
        const size_t s1 = sizeof(uint32_t) * kSelSlice;
        if ((e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)s1)) != cudaSuccess)
            return e;
        select<<<units * w.n_sel, kSelectThreads, s1, st>>>(p, c, q, seq_len, w);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        DecodeWs d = {};
        d.lse2 = w.lse2;
        d.cand = w.cand;
        d.cand_n = w.cand_n;
        d.cand2 = w.cand2;
        d.cand2_n = w.cand2_n;
        d.n_sel = w.n_sel;
        d.n_grp = w.n_grp;
        if ((e = launch_select_merge(p, d, seq_len, idx, cnt, nullptr, st)) != cudaSuccess) return e;
    } else {
        auto one = decode_quant_select_one_kernel<D, F>;
        const size_t s1 = BlockTopK::smem_bytes(Kc, kOneRound);
        if ((e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)s1)) != cudaSuccess)
            return e;
        one<<<units, kSelectThreads, s1, st>>>(p, c, q, seq_len, w, idx, cnt);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (sel)
        decode_quant_sel_scores_kernel<D, F><<<dim3(units, 8), 128, 0, st>>>(p, c, q, w.lse2, idx,
                                                                            cnt, sel);
    return cudaGetLastError();
}

}  // namespace dq

size_t decode_quant_workspace(const KParams& p) { return dq::ws_layout(p, nullptr).bytes; }

int decode_quant_kernel_count(const KParams& p, bool sel) {
    const int select = p.k - p.window > kSelMaxRanked ? 1 : sel_groups(sel_splits(p)) > 0 ? 3 : 2;
    return 2 + select + (sel ? 1 : 0);
}

cudaError_t launch_decode_quant(const KParams& p, int format, const QuantCache& c, const void* q,
                                const int32_t* seq_len, int32_t* idx, int32_t* cnt, void* o,
                                float* lse, float* sel, void* ws, cudaStream_t st) {
    if (format == HS_KV_INT4)
        return p.head_dim == 64
                   ? dq::launch_t<64, HS_KV_INT4>(p, c, q, seq_len, idx, cnt, o, lse, sel, ws, st)
                   : dq::launch_t<128, HS_KV_INT4>(p, c, q, seq_len, idx, cnt, o, lse, sel, ws, st);
    return p.head_dim == 64
               ? dq::launch_t<64, HS_KV_FP8>(p, c, q, seq_len, idx, cnt, o, lse, sel, ws, st)
               : dq::launch_t<128, HS_KV_FP8>(p, c, q, seq_len, idx, cnt, o, lse, sel, ws, st);
}

}  // namespace hs

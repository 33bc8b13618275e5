// decode_quant.cu -- decode step of the full layer over a quantised cache: it
// attends to every cached row and selects the index set of the new token, as
// decode_full.cu does over a bf16 cache.  Two kernels:
//
//  1. decode_quant_full_kernel.  The steps (32 or 16 keys) of all (sequence,
//     KV group) units, laid end to end, are cut into equal shares, one per CTA
//     of a grid that fills the GPU once: ragged batches and few long sequences
//     keep every SM busy alike.  A CTA writes one partial (m, l, O) per unit
//     that its share touches, and every 16 keys' largest logit per head.
//  2. decode_quant_select_kernel, a cluster per unit: the exact log-sum-exp
//     merge -> o, lse, then the index set.  The group score max_h (a2_h -
//     lse2_h) of a key needs every head's final lse, so it cannot be ranked in
//     pass 1.  Instead of carrying every logit over (64 bytes a key, against rows
//     of 68 or 132), the maxima bound it: a tile of 16 keys has the largest score
//     max_h (max_i a2_hi - lse2_h), exactly.  Each of the k - w best tiles (equal
//     bounds: lower tile first) holds a key at least as good as every key of the
//     others, so the k - w best keys lie in those tiles, and none is below the
//     last one's bound.  Only they are read again (at most 16 (k - w + kSlack)
//     keys), and of their keys only those that reach that bound are ranked.
//     Tiles of 32 keys: 13 us less in pass 1 (their maxima are fewer), 37 us more
//     here (32 sequences of 131072 keys, 4-bit, 16 heads: 567 + 144 us against 580 + 107).
#include <atomic>

#include "cta_select.cuh"
#include "hs_common.cuh"
#include "hs_kernels.cuh"
#include "quant_kv.cuh"

namespace hs {
namespace dq {

constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr int kMaxCtas = 640;  // partial slots reserved: at most kMaxCtas + units
template <int D, int F, int NH> using Attend = QAttend<D, F, NH, kStages>;
// Four-warp CTAs of the full kernel to an SM that the registers are divided for: 8 heads fit
// 128 registers (8-bit ragged batch, 32/8 heads: 65 us, 67 with three CTAs), 16 heads take
// 240 (a third CTA, with Q in shared memory: 581 us against 558 for 32 x 131072 keys).
// Steps of 16 keys of 128-byte rows: with 32 and three CTAs 66 us against 64.
template <int NH> constexpr int kPerSm = NH == 1 ? 4 : 2;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBoundCap = 16384;  // tile bounds a selecting CTA holds on chip
constexpr int kSub = 16;  // keys of a tile of the selection
// Tiles that may be rescored past the k - w best: the threshold is then found in fewer
// passes (one sequence of 2^20 keys 64.9 -> 62.6 us; at 64 the further tiles cost more
// than the passes, 8-bit ragged batch 52.6 -> 58.4 us).
constexpr int kSlack = 16;
// Ring of a rescoring warp (some 100 KB for the CTA's 16).
template <int D, int F> using KeyRing = QRing<D, F, false, 3>;
// Rounds of rescoring between looks at the number of candidates, where the buffer for
// that many fits (budgets k - w up to about 3000); else 1 (at the usual budgets: short
// caches 16.8 us, with a look a round 22.3; 32 x 131072 keys 104 against 112).
constexpr int kCheck = 4;

constexpr int kBitsPad = 512;     // the tiles are dealt out in chunks of 32 to up to 8 CTAs

struct Ws {
    float* part;      // [kMaxCtas + units][32 + 16 D]
    float* tmax;      // [units][tiles][16]: largest logit per head, log2 domain
    uint32_t* bits;   // [units][tiles + kBitsPad]: bounds, where a CTA's exceed kBoundCap
    int tiles;        // of a unit: t_kv in whole steps, whose tiles are all written
    size_t bytes;
};
constexpr int kMaxStep = 32;  // keys of the widest step

static Ws ws_layout(const KParams& p, void* base) {
    Ws w;
    const size_t units = (size_t)p.batch * p.hkv;
    w.tiles = ((p.t_kv - 1) / kMaxStep + 1) * (kMaxStep / kSub);
    char* c = static_cast<char*>(base);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* r = c + at;
        at += align256(bytes);
        return r;
    };
    w.part = (float*)take((kMaxCtas + units) * (32 + 16 * p.head_dim) * sizeof(float));
    w.tmax = (float*)take(units * w.tiles * 16 * sizeof(float));
    w.bits = (uint32_t*)take(w.tiles > kBoundCap ? units * (w.tiles + kBitsPad) * sizeof(uint32_t)
                                                  : 0);
    w.bytes = at;
    return w;
}

// Steps of sequence b's cache (per unit); none for a length out of range.
template <int NK>
__device__ __forceinline__ int seq_steps(const int32_t* seq_len, int b, int t_kv) {
    const int L = __ldg(seq_len + b);
    return L >= 1 && L <= t_kv ? (L - 1) / NK + 1 : 0;
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

// Reduces the maxima of a step's 16-key groups over the keys and stores them: a lane has
// V of them (group, head), and each halving of the lanes of equal t drops half of those.
// Every group of a step is stored, those past the last key too (-inf).
struct TileMaxima {
    float* at;  // this unit's [tiles][16]
    template <int NG, int NH>
    __device__ __forceinline__ void operator()(int step, const float2 (&m)[NG][NH]) const {
        constexpr int V = 2 * NG * NH;
        const int lane = threadIdx.x & 31;
        float v[V];
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                v[2 * (i * NH + n)] = m[i][n].x;
                v[2 * (i * NH + n) + 1] = m[i][n].y;
            }
        int which = 0, left = V;
#pragma unroll
        for (int bit = 16; bit >= 4; bit >>= 1) {
            left >>= 1;
            if (left > 0) {
                which = 2 * which + (lane & bit ? 1 : 0);
#pragma unroll
                for (int c = 0; c < left; ++c) {
                    const float give = lane & bit ? v[c] : v[c + left];
                    const float keep = lane & bit ? v[c + left] : v[c];
                    v[c] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, bit));
                }
            } else {
                v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
            }
        }
        const int h = 8 * ((which >> 1) % NH) + 2 * (lane & 3) + (which & 1);
        if (V == 8 || !(lane & (V == 4 ? 4 : 12)))
            at[(size_t)step * (16 * NG) + 16 * ((which >> 1) / NH) + h] = v[0];
    }
};

template <int D, int F, int NH>
__global__ void __launch_bounds__(kWarps * 32, kPerSm<NH>)
    decode_quant_full_kernel(KParams p, QuantCache cache, const __nv_bfloat16* __restrict__ q,
                             const int32_t* __restrict__ seq_len, Ws ws) {
    using A = Attend<D, F, NH>;
    constexpr int NK = A::NK;
    static_assert(kMaxStep % NK == 0, "a unit's tiles hold whole steps");
    extern __shared__ __align__(16) unsigned char smem_raw[];  // rings, reused for partials
    constexpr int kStride = A::Ring::kBytes / 4;
    static_assert(kStride >= A::kPart, "a partial fits a ring");
    float* smem = reinterpret_cast<float*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = p.group;
    const typename A::Ring ring{smem_u32(smem_raw) + warp * A::Ring::kBytes};
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
        st.init(q + ((size_t)b * p.hq + (size_t)u * g) * D, D, g, p.scale_log2);
        const QuantCache uc = unit_cache<D, F>(p, cache, unit);
        const int L = __ldg(seq_len + b);
        const TileMaxima tm{ws.tmax + (size_t)unit * ws.tiles * 16};
        if (p.bt) st.run(ring, uc, QRange<NK>{L, page_map(p, b, u)}, s0 + warp, kWarps, s1, tm);
        else st.template run_dense<kWarps>(ring, uc, L, s0 + warp, s1, tm);
        st.finish();
        st.store_part(smem + warp * kStride, g);
        __syncthreads();
        float* dst = ws.part + (size_t)(blockIdx.x + unit) * A::kPart;
        for (int e = threadIdx.x; e < g * (D / 4); e += blockDim.x) {
            const int h = e / (D / 4);
            float M = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, smem[w * kStride + 2 * h]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* pw = smem + w * kStride;
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
        __syncthreads();  // the partials are read before the rings fill again
        at += s1 - s0;
        s0 = 0;
        if (++u == p.hkv) {
            u = 0;
            do { ++b; } while (b < p.batch && (n = seq_steps<NK>(seq_len, b, p.t_kv)) == 0);
        }
    }
}

// ----------------------------------------------------------------- selection
// Shared address `a` of cluster CTA `rank`, as a generic pointer.
template <typename T>
__device__ __forceinline__ T* cluster_ptr(T* a, int rank) {
    T* r;
    asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(a), "r"(rank));
    return r;
}

// A key t such that at least k and at most k + kSlack of the distinct keys of all C CTAs
// of the cluster are >= t (fewer than k + 1 keys: the least): get(0) .. get(n - 1) are
// this CTA's.  All threads of all CTAs call; all get the result.  Range bucket select as
// cta_kth_largest, which ends as soon as the bucket that holds the k-th largest fits
// into the slack; each CTA counts its own keys and reads the others' counts.
struct ThresholdSmem {
    alignas(16) uint32_t hist[2][256];
    unsigned long long lo, hi;
    unsigned long long nlo, nhi;
    int need, done;
};
template <typename Get>
__device__ uint64_t cluster_threshold(Get get, int n, int k, ThresholdSmem& sh, int C, int rank) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    auto sync = [&] {
        __syncwarp();  // the barrier takes whole warps
        if (C > 1) cluster_sync_all();
        else __syncthreads();
    };
    uint64_t mn = ~0ull, mx = 0ull;
    for (int i = tid; i < n; i += nt) {
        const uint64_t v = get(i);
        mn = v < mn ? v : mn;
        mx = v > mx ? v : mx;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t a = shfl_xor_u64(mn, o), b = shfl_xor_u64(mx, o);
        mn = a < mn ? a : mn;
        mx = b > mx ? b : mx;
    }
    if (tid == 0) { sh.lo = ~0ull; sh.hi = 0ull; }
    for (int x = tid; x < 512; x += nt) (&sh.hist[0][0])[x] = 0u;
    __syncthreads();
    if (lane == 0 && mn <= mx) {
        atomicMin(&sh.lo, (unsigned long long)mn);
        atomicMax(&sh.hi, (unsigned long long)mx);
    }
    sync();
    uint64_t lo = ~0ull, hi = 0ull;
    for (int r = 0; r < C; ++r) {
        const ThresholdSmem* s = C > 1 ? cluster_ptr(&sh, r) : &sh;
        const uint64_t a = *(volatile const unsigned long long*)&s->lo;
        const uint64_t b = *(volatile const unsigned long long*)&s->hi;
        lo = a < lo ? a : lo;
        hi = b > hi ? b : hi;
    }
    int need = k;
    for (int pass = 0; pass < 9 && lo < hi; ++pass) {
        const int h = pass & 1, shift = max(0, top_bit64(hi - lo) - 7);
        for (int i = tid; i < n; i += nt) {
            const uint64_t v = get(i);
            if (v >= lo && v <= hi) atomicAdd(&sh.hist[h][(uint32_t)((v - lo) >> shift)], 1u);
        }
        sync();
        if (tid < 32) {
            uint32_t c[8] = {};  // lane l owns buckets 255 - 8l .. 248 - 8l, from the top
            for (int r = 0; r < C; ++r) {
                const ThresholdSmem* from = C > 1 ? cluster_ptr(&sh, r) : &sh;
                const uint4* at = reinterpret_cast<const uint4*>(&from->hist[h][248 - 8 * lane]);
                const uint4 a = at[1], b = at[0];
                const uint32_t v[8] = {a.w, a.z, a.y, a.x, b.w, b.z, b.y, b.x};
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] += v[j];
            }
            uint32_t s = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) s += c[j];
            uint32_t incl = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const uint32_t excl = incl - s;
            if (excl < (uint32_t)need && incl >= (uint32_t)need) {
                uint32_t above = excl;
                int j = 0;
                while (above + c[j] < (uint32_t)need) { above += c[j]; ++j; }
                const uint64_t nlo = lo + ((uint64_t)(255u - 8u * lane - j) << shift);
                const uint64_t span = (1ull << shift) - 1ull;
                sh.nlo = nlo;
                sh.nhi = hi - nlo < span ? hi : nlo + span;
                sh.need = need - (int)above;
                sh.done = (int)(above + c[j]) <= need + kSlack;
            }
        }
        // the other histogram was last read, by other CTAs too, before the sync above
        for (int x = tid; x < 256; x += nt) sh.hist[h ^ 1][x] = 0u;
        __syncthreads();
        lo = sh.nlo;
        hi = sh.nhi;
        need = sh.need;
        const bool done = sh.done != 0;
        __syncthreads();  // read by all before the next pass writes
        if (done) break;
    }
    sync();  // the histograms stay until all have read them
    return lo;
}

// Keys of `n` listed tiles, NK / kSub of them a step, below `end` only.
template <int NK>
struct QTiles {
    const int* tiles;
    int n, end;
    PageMap pm;
    static constexpr int kPer = NK / kSub;
    __device__ __forceinline__ int steps() const { return (n + kPer - 1) / kPer; }
    __device__ __forceinline__ bool runs() const { return kPer == 1; }
    __device__ __forceinline__ int limit() const { return end; }
    __device__ __forceinline__ int load(int step) const {
        const int i = step * kPer + (int)(threadIdx.x & (NK - 1)) / kSub;
        return i < n ? tiles[i] : -1;
    }
    __device__ __forceinline__ int key(int tile, int) const {
        if (tile < 0) return -1;
        const int k = tile * kSub + (kPer == 1 ? 0 : (int)(threadIdx.x & (kSub - 1)));
        return k < end ? k : -1;
    }
    __device__ __forceinline__ int key_at(int step, int x) const {
        return tiles[step * kPer + x / kSub] * kSub + x % kSub;
    }
};
// Keys first .. end - 1, every C-th run of NK of them from the rank-th on.
template <int NK>
struct QKeys {
    int first, end, C, rank;
    PageMap pm;
    __device__ __forceinline__ int steps() const {
        const int all = (end - first + NK - 1) / NK;
        return all > rank ? (all - rank - 1) / C + 1 : 0;
    }
    __device__ __forceinline__ bool runs() const { return true; }
    __device__ __forceinline__ int limit() const { return end; }
    __device__ __forceinline__ int load(int) const { return 0; }
    __device__ __forceinline__ int key(int, int step) const { return first + (step * C + rank) * NK; }
    __device__ __forceinline__ int key_at(int step, int x) const { return key(0, step) + x; }
};

// Rescores a source's keys, warp w of the CTA steps w, w + kSelWarps, ...: put(key,
// score, log2 domain) for each; after_rounds() by all threads, once per `check` rounds.
template <class Ring, int D, int F, int NH, class Src, class Put, class After>
__device__ __forceinline__ void score_keys(const QQuery<D, F, NH>& q, const float2 (&lse2)[NH],
                                           uint32_t ring_base, const QuantCache& c, const Src& src,
                                           int n_steps, int check, Put put, After after_rounds) {
    constexpr int NK = Ring::NK;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
    const Ring ring{ring_base + warp * Ring::kBytes};
    int ahead = warp;
    QPlace at = find<NK>(src, warp < n_steps ? src.load(warp) : 0, warp, n_steps);
    constexpr int S = Ring::kDepth;
    auto fill = [&](int s) {
        if (ahead < n_steps) ring.fill(s, c, row_of(src.pm, at), at.run);
        cp_async_commit();
        ahead += kSelWarps;
        at = find<NK>(src, ahead < n_steps ? src.load(ahead) : 0, ahead, n_steps);
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fill(i);
    int s = 0, rounds = 0;
    for (int r0 = 0; r0 < n_steps; r0 += kSelWarps) {
        const int st = r0 + warp;
        cp_async_wait<S - 2>();
        __syncwarp();
        fill(s == 0 ? S - 1 : s - 1);
        if (st < n_steps) {
            const uint32_t live = ring.live(s);
            float2 x[NK / 16][2][NH];
            q.logits(x, ring, ring.stage(s), live);
#pragma unroll
            for (int i = 0; i < NK / 16; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // the best of the quad's heads: NaN loses
                    float v = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NH; ++n)
                        v = tc::max3f(v, __fsub_rn(__fmul_rn(x[i][k][n].x, q.kf[n].x), lse2[n].x),
                                      __fsub_rn(__fmul_rn(x[i][k][n].y, q.kf[n].y), lse2[n].y));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    const int slot = 16 * i + 8 * k + (gid >> 1) + 4 * (gid & 1);
                    if (t == 0 && ((live >> slot) & 1u)) put(src.key_at(st, slot), v);
                }
        }
        s = s == S - 1 ? 0 : s + 1;
        if (++rounds == check) {
            rounds = 0;
            after_rounds();
        }
    }
    cp_async_wait<0>();
    __syncwarp();
}

// Keeps the K largest of buf[0..n) (n > K), in buf[0..K); tmp holds K keys.
__device__ void keep_largest(uint64_t* buf, int n, int K, uint64_t* tmp, CtaSelectSmem& cs,
                             int* s_n, uint64_t* kth_out) {
    const uint64_t kth = cta_kth_largest([&](int i) { return buf[i]; }, n, K, cs);
    if (threadIdx.x == 0) *s_n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (buf[i] >= kth) tmp[atomicAdd(s_n, 1)] = buf[i];
    __syncthreads();
    for (int i = threadIdx.x; i < K; i += blockDim.x) buf[i] = tmp[i];
    __syncthreads();
    *kth_out = kth;
}

// Ascending sort of a[0 .. n), n a power of two up to 4096, by kSelThreads threads: bitonic;
// exchanges within a warp's 64 values stay in registers (of 55 steps for 1024
// values 10 go through shared memory).
__device__ void sort_ascending(uint64_t* a, int n) {
    const int lane = threadIdx.x & 31;
    for (int base = threadIdx.x - lane; base * 2 < n; base += kSelThreads) {
        // a warp's 64 values, two a lane (i and i + 32)
        uint64_t* w = a + base * 2;
        uint64_t x = base * 2 + lane < n ? w[lane] : ~0ull;
        uint64_t y = base * 2 + lane + 32 < n ? w[lane + 32] : ~0ull;
        warp_sort64(x, y);
        const bool down = (base * 2) & 64;  // alternate runs of 64 descend
        if (base * 2 + lane < n) w[down ? 63 - lane : lane] = x;
        if (base * 2 + lane + 32 < n) w[down ? 31 - lane : lane + 32] = y;
    }
    __syncthreads();
    for (int k = 128; k <= n; k <<= 1) {
        int j = k >> 1;
        for (; j >= 64; j >>= 1) {
            for (int i = threadIdx.x; i < n / 2; i += kSelThreads) {
                const int p = 2 * i - (i & (j - 1)), q = p + j;
                const uint64_t x = a[p], y = a[q];
                if ((x > y) == ((p & k) == 0)) { a[p] = y; a[q] = x; }
            }
            __syncthreads();
        }
        for (int base = threadIdx.x - lane; base * 2 < n; base += kSelThreads) {
            uint64_t* w = a + base * 2;
            uint64_t x = w[lane], y = w[lane + 32];
            const bool up = ((base * 2) & k) == 0;
            if ((x > y) == up) { const uint64_t z = x; x = y; y = z; }
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) {
                const uint64_t px = shfl_xor_u64(x, s), py = shfl_xor_u64(y, s);
                const bool low = ((lane & s) == 0) == up;  // keeps the smaller
                x = low == (x < px) ? x : px;
                y = low == (y < py) ? y : py;
            }
            w[lane] = x;
            w[lane + 32] = y;
        }
        __syncthreads();
    }
}

// Dynamic shared memory of the selection, for Kc = k - w.
template <int D, int F>
struct SelSmem {
    static constexpr size_t most(size_t a, size_t b) { return a > b ? a : b; }
    static constexpr size_t kFront =  // rings; before that, tile bounds or the merge's sums
        most(kSelWarps * (size_t)KeyRing<D, F>::kBytes, sizeof(uint32_t) * kBoundCap);
    static constexpr int kRound = kSelWarps * KeyRing<D, F>::NK;  // keys of a round, at most
    __host__ __device__ static int cap(int Kc, int check) { return 2 * Kc + check * kRound; }
    __host__ __device__ static int sort_n(int Kc) { return next_pow2(Kc > 0 ? Kc : 1); }
    __host__ __device__ static size_t bytes(int Kc, int check) {
        return kFront + sizeof(uint64_t) * (cap(Kc, check) + sort_n(Kc)) + sizeof(int) * (Kc + 2 + kSlack);
    }
    static constexpr size_t kMost = 232448 - 4096;  // a CTA's shared memory, less the static part
    static int check(int Kc) { return bytes(Kc, kCheck) <= kMost ? kCheck : 1; }
};

template <int D, int F, int NH>
__global__ void __launch_bounds__(kSelThreads, 1)
    decode_quant_select_kernel(KParams p, QuantCache cache, const __nv_bfloat16* __restrict__ q,
                               const int32_t* __restrict__ seq_len, Ws ws, int grid1, int C, int check,
                               __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                               int32_t* __restrict__ idx, int32_t* __restrict__ cnt,
                               float* __restrict__ sel) {
    using A = Attend<D, F, NH>;
    using S = SelSmem<D, F>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ CtaSelectSmem cs;
    __shared__ ThresholdSmem ts;
    __shared__ float s_m[16], s_lse2[16];
    __shared__ int s_n, s_list, s_cut;
    __shared__ unsigned long long s_thr;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane & 3, g = p.group;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int unit = blockIdx.x / C, u = unit % p.hkv, b = unit / p.hkv;
    const int L = __ldg(seq_len + b);
    const size_t head0 = (size_t)b * p.hq + (size_t)u * g;
    int32_t* irow = idx + (size_t)unit * p.ksel;
    float* srow = sel ? sel + (size_t)unit * p.ksel : nullptr;
    const int n = seq_steps<A::NK>(seq_len, b, p.t_kv);
    if (n == 0) {  // length out of range: nothing attended, nothing selected
        if (rank != 0) return;
        for (int x = tid; x < g * D; x += blockDim.x) o[head0 * D + x] = __float2bfloat16_rn(0.f);
        for (int x = tid; x < g; x += blockDim.x) lse[head0 + x] = -INFINITY;
        for (int x = tid; x < p.ksel; x += blockDim.x) {
            irow[x] = -1;
            if (srow) srow[x] = 0.f;
        }
        if (tid == 0) { cnt[unit] = 0; set_status(HS_ERR_BOUNDS); }
        return;
    }
    // ---- merge of the unit's partials
    if (tid < 16) s_lse2[tid] = INFINITY;  // heads past the group never score
    __syncthreads();
    {
        const long long before = sum_steps<A::NK>(seq_len, 0, b, p.t_kv);
        const long long total = (before + sum_steps<A::NK>(seq_len, b, p.batch, p.t_kv)) * p.hkv;
        const long long first = before * p.hkv + (long long)u * n;
        const int G = ctas_used(grid1, total);
        const int c0 = share_of(first, G, total), parts = share_of(first + n - 1, G, total) - c0 + 1;
        const float* base = ws.part + (size_t)(c0 + unit) * A::kPart;
        if (warp < g) {
            float M = -INFINITY, l = 0.f;
            for (int c = lane; c < parts; c += 32) M = fmaxf(M, base[(size_t)c * A::kPart + 2 * warp]);
            M = warp_max(M);
            for (int c = lane; c < parts; c += 32) {
                const float* pc = base + (size_t)c * A::kPart + 2 * warp;
                l += pc[1] * sq::merge_weight(pc[0], M);
            }
            l = warp_sum(l);
            if (lane == 0) {
                const float l2 = l == 0.f ? -INFINITY : M + log2f(l);
                s_m[warp] = M;
                s_lse2[warp] = l2;
                if (warp % C == rank) lse[head0 + warp] = l2 * kLn2;
            }
        }
        __syncthreads();
        // heads rank, rank + C, ...: each float4 of their outputs by `per` threads
        const int heads = (g - rank + C - 1) / C, items = max(0, heads) * (D / 4);
        float4* red = reinterpret_cast<float4*>(smem_raw);  // [kSelThreads]
        int per = 1;
        while (2 * per * items <= kSelThreads && per < parts) per *= 2;
        for (int i0 = 0; i0 < items; i0 += kSelThreads / per) {
            const int it = i0 + tid / per, pr = tid % per;
            const int h = (it / (D / 4)) * C + rank, d4 = it % (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (it < items) {
                const float M = s_m[h];
#pragma unroll 4
                for (int c = pr; c < parts; c += per) {
                    const float* pc = base + (size_t)c * A::kPart;
                    const float f = sq::merge_weight(pc[2 * h], M);
                    const float4 x = reinterpret_cast<const float4*>(pc + 32 + h * D)[d4];
                    acc.x += x.x * f;
                    acc.y += x.y * f;
                    acc.z += x.z * f;
                    acc.w += x.w * f;
                }
            }
            red[tid] = acc;
            __syncthreads();
            if (it < items && pr == 0) {
                for (int x = 1; x < per; ++x) {
                    const float4 y = red[tid + x];
                    acc.x += y.x;
                    acc.y += y.y;
                    acc.z += y.z;
                    acc.w += y.w;
                }
                // sum p = 2^(lse2 - M); no key: both sums are 0
                const float inv = s_m[h] == -INFINITY && acc.x == 0.f ? 0.f : exp2f(s_m[h] - s_lse2[h]);
                *reinterpret_cast<uint2*>(o + (head0 + h) * D + 4 * d4) = make_uint2(
                    pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            }
            __syncthreads();
        }
    }
    // ---- the index set
    const int Kc = p.k - p.window;
    const bool ranked = L > p.k && Kc > 0;
    const int lo = L > p.k ? L - p.window : 0;  // keys lo.. are all selected
    if (!ranked && rank != 0) return;
    const QuantCache uc = unit_cache<D, F>(p, cache, unit);
    const PageMap pm = page_map(p, b, u);
    uint64_t* buf = reinterpret_cast<uint64_t*>(smem_raw + S::kFront);  // [cap(Kc)]
    uint64_t* tmp = buf + S::cap(Kc, check);                                    // [sort_n(Kc)]
    int* list = reinterpret_cast<int*>(tmp + S::sort_n(Kc));             // [Kc + 2 + kSlack]
    QQuery<D, F, NH> qq;
    float2 nl[NH];
    if (ranked || srow) {
        qq.init(q + head0 * D, D, g, p.scale_log2);
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const int h = 8 * n + 2 * t;
            nl[n] = make_float2(s_lse2[h], s_lse2[h + 1]);
        }
    }
    if (tid == 0) { s_n = 0; s_list = 0; s_thr = 0ull; }
    __syncthreads();
    int n_best = 0;
    if (ranked) {
        const int full = lo / kSub;  // tiles of ranked keys only; tile `full` has some if lo % kSub
        // this CTA's tiles: chunks of 32, dealt out over the cluster
        const int chunks = (full + 31) / 32;
        const int mine = (chunks > rank ? (chunks - rank - 1) / C + 1 : 0) * 32 -
                         ((chunks - 1) % C == rank ? chunks * 32 - full : 0);
        auto tile = [&](int i) { return ((i >> 5) * C + rank) * 32 + (i & 31); };
        auto offer = [&](int key, float v) {
            const uint64_t c = sel_key(v, (uint32_t)key);
            if (c >= s_thr) buf[atomicAdd(&s_n, 1)] = c;
        };
        const int cap = S::cap(Kc, check);
        auto look = [&] {
            __syncthreads();
            const int have = s_n;
            __syncthreads();  // read by all before the next offers
            if (have > cap - check * S::kRound) {
                uint64_t kth;
                keep_largest(buf, have, Kc, tmp, cs, &s_cut, &kth);
                if (tid == 0) { s_thr = kth; s_n = Kc; }
                __syncthreads();
            }
        };
        if (full <= Kc) {  // no tile can be left out
            using Ring = KeyRing<D, F>;
            const QKeys<Ring::NK> src{0, lo, C, rank, pm};
            score_keys<Ring, D, F, NH>(qq, nl, smem_u32(smem_raw), uc, src, src.steps(), check, offer, look);
        } else {
            const float4* tm = reinterpret_cast<const float4*>(ws.tmax + (size_t)unit * ws.tiles * 16);
            uint32_t* bits = mine <= kBoundCap ? reinterpret_cast<uint32_t*>(smem_raw)
                                               : ws.bits + (size_t)unit * (ws.tiles + kBitsPad) +
                                                     (size_t)rank * ((chunks + C - 1) / C) * 32;
            constexpr int U = 2, Q4 = 2 * NH;  // tiles in flight per thread, float4 of a tile
            for (int i0 = tid; i0 < mine; i0 += U * kSelThreads) {
                float4 a[U][Q4];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int i = i0 + k * kSelThreads, x = tile(i);
#pragma unroll
                    for (int q4 = 0; q4 < Q4; ++q4)
                        a[k][q4] = i < mine ? __ldg(tm + (size_t)x * 4 + q4)
                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int i = i0 + k * kSelThreads;
                    if (i >= mine) break;
                    float v = -INFINITY;
#pragma unroll
                    for (int q4 = 0; q4 < Q4; ++q4) {
                        const float av[4] = {a[k][q4].x, a[k][q4].y, a[k][q4].z, a[k][q4].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v = fmaxf(v, __fsub_rn(av[e], s_lse2[4 * q4 + e]));
                    }
                    bits[i] = float_order(v);
                }
            }
            __syncthreads();
            auto key = [&](int i) -> uint64_t {
                return ((uint64_t)bits[i] << 32) | (uint64_t)(0xffffffffu - (uint32_t)tile(i));
            };
            const uint64_t kth = cluster_threshold(key, mine, Kc, ts, C, rank);
            for (int i = tid; i < mine; i += blockDim.x)
                if (key(i) >= kth) list[atomicAdd(&s_list, 1)] = tile(i);
            if (tid == 0) {
                // the bounds and the scores below are the same arithmetic on the same
                // operands; the step down covers a difference in their last bits.  kth may
                // lie between two keys, and stand for no number.
                const float th = sel_key_score(kth);
                float mag = fabsf(th);
                for (int h = 0; h < g; ++h) mag = fmaxf(mag, fabsf(s_lse2[h]));
                s_thr = isfinite(th) && isfinite(mag) ? (uint64_t)float_order(th - 4e-6f * mag) << 32 : 0ull;
            }
            __syncthreads();
            if (tid == 0 && rank == 0 && lo % kSub != 0) list[s_list++] = full;
            __syncthreads();
            using Ring = KeyRing<D, F>;
            const QTiles<Ring::NK> src{list, s_list, lo, pm};
            score_keys<Ring, D, F, NH>(qq, nl, smem_u32(smem_raw), uc, src, src.steps(), check, offer, look);
        }
        __syncthreads();
        n_best = s_n;
        uint64_t kth;
        if (n_best > Kc) {
            keep_largest(buf, n_best, Kc, tmp, cs, &s_cut, &kth);
            n_best = Kc;
        }
        if (C > 1) {
            if (tid == 0) s_n = n_best;
            __syncwarp();
            cluster_sync_all();
            if (rank == 0) {
                for (int r = 1; r < C; ++r) {
                    const int m = *(volatile int*)cluster_ptr(&s_n, r);  // up to Kc
                    if (n_best + m > cap) {
                        __syncthreads();
                        keep_largest(buf, n_best, Kc, tmp, cs, &s_cut, &kth);
                        n_best = Kc;
                    }
                    const uint64_t* from = cluster_ptr(buf, r);
                    for (int x = tid; x < m; x += blockDim.x) buf[n_best + x] = from[x];
                    n_best += m;
                }
                __syncthreads();
                if (n_best > Kc) {
                    keep_largest(buf, n_best, Kc, tmp, cs, &s_cut, &kth);
                    n_best = Kc;
                }
            }
            __syncwarp();
            cluster_sync_all();  // the others keep their buffers until here
            if (rank != 0) return;
        }
        const int sort_n = next_pow2(max(n_best, 1));
        for (int x = tid; x < sort_n; x += blockDim.x)
            tmp[x] = x < n_best ? ((uint64_t)sel_key_id(buf[x]) << 32) | (buf[x] >> 32) : ~0ull;
        __syncthreads();
        sort_ascending(tmp, sort_n);
        for (int x = tid; x < n_best; x += blockDim.x) {
            irow[x] = (int32_t)(tmp[x] >> 32);
            if (srow) srow[x] = exp2f(order_float((uint32_t)tmp[x]));
        }
    }
    for (int x = tid; x < L - lo; x += blockDim.x) {
        irow[n_best + x] = lo + x;
        if (srow) srow[n_best + x] = 0.f;  // keys on bad pages get no score below
    }
    const int n_out = n_best + L - lo;
    for (int x = n_out + tid; x < p.ksel; x += blockDim.x) {
        irow[x] = -1;
        if (srow) srow[x] = 0.f;
    }
    if (tid == 0) cnt[unit] = n_out;
    if (srow) {
        __syncthreads();
        using Ring = KeyRing<D, F>;
        const QKeys<Ring::NK> src{lo, L, 1, 0, pm};
        score_keys<Ring, D, F, NH>(
            qq, nl, smem_u32(smem_raw), uc, src, src.steps(), 1,
            [&](int key, float v) { srow[n_best + key - lo] = exp2f(v); }, [] {});
    }
}

// CTAs of the full kernel that fill the current device once, and its SMs
// (cached per device).
template <int D, int F, int NH>
static cudaError_t full_grid(size_t smem, int* ctas, int* sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        int per = 0;
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                 &per, decode_quant_full_kernel<D, F, NH>, kWarps * 32, smem)) != cudaSuccess)
            return e;
        n = min(kMaxCtas, max(1, per) * *sms);
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *ctas = n;
    return cudaSuccess;
}

template <int D, int F, int NH>
static cudaError_t launch_t(const KParams& p, const QuantCache& c, const void* q_,
                            const int32_t* seq_len, int32_t* idx, int32_t* cnt, void* o,
                            float* lse, float* sel, void* ws_, cudaStream_t st) {
    using A = Attend<D, F, NH>;
    const __nv_bfloat16* q = (const __nv_bfloat16*)q_;
    const Ws w = ws_layout(p, ws_);
    const int units = p.batch * p.hkv;
    cudaError_t e;
    auto full = decode_quant_full_kernel<D, F, NH>;
    const size_t smem = (size_t)kWarps * A::Ring::kBytes;
    if ((e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
        cudaSuccess)
        return e;
    int G = 0, sms = 148;
    if ((e = full_grid<D, F, NH>(smem, &G, &sms)) != cudaSuccess) return e;
    // no CTA below a step per warp, as far as the capacity tells
    const int steps = (p.t_kv + A::NK - 1) / A::NK;
    G = (int)max(1ll, min((long long)G, ((long long)units * steps + kWarps - 1) / kWarps));
    full<<<G, kWarps * 32, smem, st>>>(p, c, q, seq_len, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    auto select = decode_quant_select_kernel<D, F, NH>;
    const int check = SelSmem<D, F>::check(p.k - p.window);
    const size_t s1 = SelSmem<D, F>::bytes(p.k - p.window, check);
    if ((e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s1)) !=
        cudaSuccess)
        return e;
    // Clusters as wide as a wave of one CTA per SM allows, while the capacity gives a CTA
    // more than 256 steps (one sequence of 2^20 keys: 64 us on 4 x 8 CTAs, 244 on 4; 8-bit
    // ragged batch of 9 x 8 units: 55 us on pairs, 70 alone).
    int C = 1;
    while (C < 8 && units * C * 2 <= sms && steps / (C * 2) > 256) C *= 2;
    cudaLaunchConfig_t cfg = {};
    // Its launch overlaps the end of the full kernel, for whose results it waits first
    // (a step over short caches 29.1 -> 28.0 us, 8-bit ragged batch 123.0 -> 121.5; an
    // earlier signal from the full kernel gains no more, and costs long caches 1-4 us).
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(units * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = s1;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, select, p, c, q, seq_len, w, G, C, check, (__nv_bfloat16*)o, lse, idx,
                              cnt, sel);
}

struct Launch {
    const KParams& p;
    const QuantCache& c;
    const void* q;
    const int32_t* seq_len;
    int32_t *idx, *cnt;
    void* o;
    float *lse, *sel;
    void* ws;
    cudaStream_t st;
    template <int D, int F, int NH>
    cudaError_t operator()() const {
        return launch_t<D, F, NH>(p, c, q, seq_len, idx, cnt, o, lse, sel, ws, st);
    }
};

}  // namespace dq

size_t decode_quant_workspace(const KParams& p) { return dq::ws_layout(p, nullptr).bytes; }

cudaError_t launch_decode_quant(const KParams& p, int format, const QuantCache& c, const void* q,
                                const int32_t* seq_len, int32_t* idx, int32_t* cnt, void* o,
                                float* lse, float* sel, void* ws, cudaStream_t st) {
    return sq::dispatch(p, format, dq::Launch{p, c, q, seq_len, idx, cnt, o, lse, sel, ws, st});
}

}  // namespace hs

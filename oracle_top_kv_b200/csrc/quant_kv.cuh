// quant_kv.cuh -- rows of a quantised K^F/V^F cache: their storage, and
// attention over them with the codes as matrix operands.
//
// A stored row is head_dim codes plus one 4-byte entry {scale, zero} (bf16
// each); code c stands for scale * c + zero.  HS_KV_INT4: c = 0..15, element
// 2j in the low and 2j + 1 in the high nibble of byte j.  HS_KV_FP8: c is an
// e4m3 number, one byte per element.
//
// Attention never rebuilds the values.  For a key with entry (s, z),
//     scale q.k^ = scale (s (q.c) + z sum(q)),
//     sum_i p_i v^_i = sum_i (p_i s_i) c_i + sum_i p_i z_i:
// both products run on the codes, exact in fp16, with fp32 accumulators
// (mma.m16n8k16), and scale and zero are applied to the logits, to P and to one
// running sum per head.  fp16 rather than bf16, because codes reach it in few
// instructions: a 4-bit code in the lowest bits of a half is the number c 2^-24, four
// bits higher 16 c 2^-24, both exact subnormals, so 8 codes take a shift and four ANDs
// (the factor 16 of odd elements is taken from q and from the outputs; against the
// conversion from e4m3 below, which takes seven instructions: 32 sequences of 131072
// keys, 16 heads, 578 -> 538 us; the error of a logit grew from 2e-6 to 5e-6 at 23);
// 8-bit codes are converted in pairs.  What fp16's range needs:
//  - q is scaled by a power of two per head so that max|q| lies in [2^14, 2^15);
//    a bf16 element is then exact unless it is 2^-25 of the largest or less
//    (error 2^-35 of the largest);
//  - p_i s_i is taken relative to 2^10 at the running maximum (growing to
//    2^14 before O is rescaled) and to a power of two above the largest |s_i|
//    seen, and rounded to fp16: relative 2^-12 for weights down to 2^-24 of the
//    largest, an absolute 2^-35 of it below (and in 4 bits the zero points are
//    weighted by the rounded numbers too, QAttend::centre).
// Everything else is fp32.  The kernels are bound by what a scheduler gets issued, not by
// memory: 16 keys of 128 dims and 16 heads take 294 instructions, 32 of them MMAs, in some
// 590 cycles at two warps a scheduler (issue active 50%, top stall a fixed-latency wait,
// DRAM 49%).  An MMA alone takes 8.7 cycles of its scheduler; each FFMA beside it adds one,
// up to three LOP3s 0.6 each (a fourth 1.6), so that 278 cycles go to the MMAs and the
// others overlap them in part; how much is lost to the few warps is not settled.
// (32 sequences of 131072 keys, 16 heads of 128: 569 us, 4.0 TB/s of cache.)
//
// One warp takes 16 keys at a time: they are the rows of S^T = K Q^T, 8 heads at a
// time its columns, and O^T = V^T P^T has 16 dimensions at a time as rows (P^T's
// fragments from movmatrix), so that groups of up to 8 heads need half the MMAs of 16.
// Lane (gid, t) of the warp (gid = lane / 4, t = lane % 4) needs of a key's K row the
// t-th quarter and of a V row the gid-th eighth (Q's fragments take the same
// order of dimensions), so rows are read from shared memory as they lie in the
// cache.  cp.async fills a ring of stages per warp; it also places the rows:
// within 16 keys, key t + 4 e + 8 j is row 2 t + e of the j-th 8 rows; K rows lie in
// that order, V rows keep their own with 16-byte chunks swizzled, and the four entries
// of equal t are adjacent: every shared read of rows is free of bank conflicts.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attend_mma.cuh"
#include "hs_common.cuh"
#include "hs_kernels.cuh"
#include "tc_ptx.cuh"

namespace hs {

// A quantised cache: codes and {scale, zero} entries, rows contiguous per
// (sequence, kv head), or per (page, kv head) with KParams' block table.
struct QuantCache {
    const uint8_t* kc;
    const uint32_t* ks;
    const uint8_t* vc;
    const uint32_t* vs;
};

template <int D, int F>
struct QRow {
    static constexpr int kBytes = F == HS_KV_INT4 ? D / 2 : D;
    static constexpr int kKW = kBytes / 16;  // words of a quarter row
    static constexpr int kVW = kBytes / 32;  // words of an eighth row
};

__device__ __forceinline__ float entry_scale(uint32_t e) { return __uint_as_float(e << 16); }
__device__ __forceinline__ float entry_zero(uint32_t e) { return __uint_as_float(e & 0xffff0000u); }

// D = A(16x16 fp16, row) * B(16x8 fp16, col) + D (fp32)
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The e4m3 pairs in the low and in the high half of x as fp16 pairs (exact).
__device__ __forceinline__ void e4m3_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

// What a code of 1 counts for in the operands; a 4-bit code of an odd element for 16 times
// that.
template <int F> constexpr float kCodeUnit = F == HS_KV_INT4 ? 1.f / 16777216.f : 1.f;
template <int F>
__host__ __device__ constexpr float odd_unit(int odd) { return F == HS_KV_INT4 && odd ? 1.f / 16.f : 1.f; }

// Dimension (of a quarter row) that element e (0: b0 low, 1: b0 high, 2: b1
// low, 3: b1 high) of k step `ks` holds.
template <int F>
__host__ __device__ constexpr int k_dim(int ks, int e) {
    return F == HS_KV_INT4 ? 8 * (ks >> 1) + (ks & 1) + 4 * (e & 1) + (e & 2) : 4 * ks + e;
}

// B fragment (b0, b1) of k step `ks` from a lane's quarter of a K row.
template <int F, int N>
__device__ __forceinline__ void k_frag(const uint32_t (&w)[N], int ks, uint32_t& b0, uint32_t& b1) {
    if constexpr (F == HS_KV_INT4) {
        const uint32_t mask = ks & 1 ? 0x00f000f0u : 0x000f000fu;
        b0 = w[ks >> 1] & mask;
        b1 = (w[ks >> 1] >> 8) & mask;
    } else {
        e4m3_f16(w[ks], b0, b1);
    }
}

// Pairs (a[j + i], b[j + i]), i = 0..3, of a lane's eighths of two V rows, j a
// multiple of 4.
template <int F, int N>
__device__ __forceinline__ void v_pairs(const uint32_t (&a)[N], const uint32_t (&b)[N], int j,
                                        uint32_t (&p)[4]) {
    if constexpr (F == HS_KV_INT4) {
        // two neighbouring bytes of each row
        const uint32_t x = __byte_perm(a[j >> 3], b[j >> 3], (j & 4) ? 0x7632 : 0x5410);
        const uint32_t y = x >> 8;
        p[0] = x & 0x000f000fu;
        p[1] = x & 0x00f000f0u;
        p[2] = y & 0x000f000fu;
        p[3] = y & 0x00f000f0u;
    } else {
        e4m3_f16(__byte_perm(a[j >> 2], b[j >> 2], 0x5140), p[0], p[1]);
        e4m3_f16(__byte_perm(a[j >> 2], b[j >> 2], 0x7362), p[2], p[3]);
    }
}

// ------------------------------------------------------------- row sources
// A source says which keys a warp's steps of NK slots hold, in two parts, so that what the
// first one loads is not needed at once:
//   load(step): a word that the lane needs for it (an index entry, a tile);
//   key(word, step): the logical key of the lane's slot, -1 if that slot is masked or
//     out of range; where runs() holds, of the step's first slot: the step's slots are
//     consecutive keys, of which those below limit() count.
// `pm`: where keys lie; pm.bt null: a contiguous cache, key = row.

// Logical keys 0 .. n - 1.
template <int NK>
struct QRange {
    int n;
    PageMap pm;
    __device__ __forceinline__ bool runs() const { return true; }
    __device__ __forceinline__ int limit() const { return n; }
    __device__ __forceinline__ int load(int) const { return 0; }
    __device__ __forceinline__ int key(int, int step) const { return step * NK; }
};
// Entries of an index row (token mode, B = 1: keys; block mode: blocks clipped to
// keys <= t).
template <int NK>
struct QIndex {
    const int32_t* ids;
    int n, B, t, top;
    uint32_t per, inv;  // where runs(): steps of a block, and 2^32 / per rounded up
    PageMap pm;
    __device__ __forceinline__ QIndex(const int32_t* ids_, int n_, int B_, int t_, const PageMap& pm_)
        : ids(ids_), n(n_), B(B_), t(t_), top(t_ / B_), pm(pm_) {
        per = B % NK == 0 ? B / NK : 0;
        inv = per > 1 ? 0xffffffffu / per + 1 : 0;
    }
    __device__ __forceinline__ bool runs() const { return per != 0; }
    __device__ __forceinline__ int limit() const { return t + 1; }
    // the block of a run's step (exact for steps < 2^32 / per)
    __device__ __forceinline__ uint32_t block(int step) const {
        return per == 1 ? step : __umulhi(step, inv);
    }
    __device__ __forceinline__ int slot(int step) const {
        return step * NK + (int)(threadIdx.x & (NK - 1));
    }
    __device__ __forceinline__ int load(int step) const {
        if (runs()) return step * NK < n ? __ldg(ids + block(step)) : 0;
        const int s = slot(step);
        return s < n ? __ldg(ids + (B == 1 ? s : s / B)) : 0;
    }
    __device__ __forceinline__ int key(int id, int step) const {
        if (!runs() && slot(step) >= n) return -1;
        if (id < 0 || id > top) { set_status(HS_ERR_BOUNDS); return -1; }
        if (B == 1) return id;
        const int k = id * B + (runs() ? (int)(step - block(step) * per) * NK : slot(step) % B);
        return k <= t ? k : -1;
    }
};
// A step's keys found: a row (contiguous cache) or an offset in page `page`; the first
// one's for a run.  -1: none.
struct QPlace {
    int at, page;
    bool run;
};
template <int NK, class Src>
__device__ __forceinline__ QPlace find(const Src& src, int word, int step, int n_steps) {
    QPlace p{-1, 0, false};
    if (step >= n_steps) return p;
    int k = src.key(word, step);
    if (src.runs() && k >= 0) {
        p.run = k + NK <= src.limit();
        if (src.pm.bt) p.run = p.run && src.pm.page_size % NK == 0 && k % NK == 0;
        if (!p.run) {
            k += threadIdx.x & (NK - 1);
            if (k >= src.limit()) k = -1;
        }
    }
    if (src.pm.bt && k >= 0) {
        const int lp = k / src.pm.page_size;
        p.page = lp < src.pm.max_pages ? __ldg(src.pm.bt + lp) : -1;
        k -= lp * src.pm.page_size;
    }
    p.at = k;
    return p;
}
// The row, relative to the warp's bases, -1 if none or on a bad page.
__device__ __forceinline__ int row_of(const PageMap& pm, const QPlace& p) {
    if (!pm.bt || p.at < 0) return p.at;
    if (p.page < 0 || p.page >= pm.n_pages) { set_status(HS_ERR_BOUNDS); return -1; }
    return (p.page * pm.hkv + pm.u) * pm.page_size + p.at;
}

// -------------------------------------------------------------- ring of rows
// A warp's stages.  K only: the V half is neither filled nor reserved.
template <int D, int F, bool kV, int kStages, int kKeys = QRow<D, F>::kBytes <= 64 ? 32 : 16>
struct QRing {
    using R = QRow<D, F>;
    static constexpr int RB = R::kBytes;
    static constexpr int NK = kKeys, kDepth = kStages;   // keys of a stage; stages
    static constexpr int kKeyBytes = NK * RB, kHalf = kKeyBytes + NK * 4;
    static constexpr int kStage = kHalf * (kV ? 2 : 1);  // codes, entries; K, then V
    static constexpr int kBytes = kStages * (kStage + 16);
    static constexpr int CH = RB / 16;                   // 16-byte chunks of a row

    uint32_t base;  // shared address, 16-byte aligned
    // the lane's places in a stage: what it reads, and where its copies go
    uint32_t k_at, v_at, e_at, k_to, v_to, e_to;

    __device__ __forceinline__ explicit QRing(uint32_t at) : base(at) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
        const int row = lane / CH, ch = lane % CH;
        constexpr int PER = 16 / (RB / 8) > 0 ? 16 / (RB / 8) : 1;  // eighths per chunk
        k_at = (uint32_t)(gid * RB + (RB == 128 ? ((2 * t) ^ (gid & 1)) << 4 : t * (RB / 4)));
        v_at = (uint32_t)(kHalf + v_slot(t, gid / PER) + (gid % PER) * (RB / 8));
        e_at = (uint32_t)(kKeyBytes + 16 * (gid >> 1) + 4 * (gid & 1));
        k_to = k_slot(row, ch);
        v_to = kHalf + v_slot(row, ch);
        e_to = (uint32_t)(kKeyBytes + 4 * ((lane & ~15) + 4 * (lane & 3) + ((lane >> 2) & 3)));
    }
    __device__ __forceinline__ uint32_t stage(int s) const { return base + (uint32_t)s * kStage; }
    __device__ __forceinline__ uint32_t mask_at(int s) const {
        return base + kStages * kStage + 16u * s;
    }
    __device__ static __forceinline__ uint32_t k_slot(int key, int c) {
        const int n = (key & ~7) + 2 * (key & 3) + ((key >> 2) & 1);
        return (uint32_t)(n * RB + ((RB == 128 ? c ^ (n & 1) : c) << 4));
    }
    __device__ static __forceinline__ uint32_t v_slot(int key, int c) {
        const int x = RB == 128 ? (key & 3) << 1 : RB == 64 ? key & 2 : 0;
        return (uint32_t)(key * RB + ((c ^ x) << 4));
    }
    // K place of row lane / CH + i * PASS, from that of row lane / CH: PASS rows are
    // 512 bytes; of 128-byte rows, 4 of them are half a tile, whose rows are the odd ones.
    static constexpr int PASS = 32 / CH;
    __device__ __forceinline__ uint32_t k_dst(int i) const {
        if constexpr (RB == 128) return (i & 1 ? (k_to ^ 16u) + 128u : k_to) + (uint32_t)(i >> 1) * 1024u;
        else return k_to + (uint32_t)i * 512u;
    }

    // Starts the copies of a step.
    // row: the lane's, or the first one's of a run (-1: a run on a bad page).
    __device__ __forceinline__ void fill(int s, const QuantCache& c, int row, bool run) const {
        const int lane = threadIdx.x & 31;
        const uint32_t st = stage(s);
        uint32_t live = 0xffffffffu;
        if (run && row >= 0) {  // consecutive bytes
            const uint8_t* kp = c.kc + (size_t)row * RB + lane * 16;
            const uint8_t* vp = c.vc + (size_t)row * RB + lane * 16;
#pragma unroll
            for (int i = 0; i < NK / PASS; ++i) {
                copy16(st + k_dst(i), kp + i * 512);
                if constexpr (kV) copy16(st + v_to + i * 512, vp + i * 512);
            }
            if (NK == 32 || lane < NK) {
                copy4(st + e_to, c.ks + (size_t)row + lane);
                if constexpr (kV) copy4(st + kHalf + e_to, c.vs + (size_t)row + lane);
            }
        } else if ((live = __ballot_sync(0xffffffffu, row >= 0)) == 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < NK / PASS; ++i) {
                const uint32_t r = __shfl_sync(0xffffffffu, row, lane / CH + i * PASS);
                const size_t off = (size_t)r * RB + (lane % CH) * 16;
                copy16(st + k_dst(i), c.kc + off);
                if constexpr (kV) copy16(st + v_to + i * 512, c.vc + off);
            }
            if (NK == 32 || lane < NK) {
                copy4(st + e_to, c.ks + (uint32_t)row);
                if constexpr (kV) copy4(st + kHalf + e_to, c.vs + (uint32_t)row);
            }
        } else {  // rows that do not count are zeros
#pragma unroll
            for (int i = 0; i < NK / PASS; ++i) {
                const int r = __shfl_sync(0xffffffffu, row, lane / CH + i * PASS);
                const size_t off = r >= 0 ? (size_t)r * RB + (lane % CH) * 16 : 0;
                cp_async16(st + k_dst(i), c.kc + off, r >= 0);
                if constexpr (kV) cp_async16(st + v_to + i * 512, c.vc + off, r >= 0);
            }
            if (NK == 32 || lane < NK) {
                const size_t off = row >= 0 ? (size_t)row : 0;
                cp_async4(st + e_to, c.ks + off, row >= 0);
                if constexpr (kV) cp_async4(st + kHalf + e_to, c.vs + off, row >= 0);
            }
        }
        if (lane == 0)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(mask_at(s)), "r"(live) : "memory");
    }
    // The same of NK consecutive rows, given the lane's 16 bytes and entry of the first
    // rows; `to`: offset of the stage.
    __device__ __forceinline__ void fill_dense(uint32_t to, const uint8_t* kp, const uint8_t* vp,
                                               const uint32_t* ke, const uint32_t* ve) const {
        const uint32_t st = base + to;
#pragma unroll
        for (int i = 0; i < NK / PASS; ++i) {
            copy16(st + k_dst(i), kp + i * 512);
            if constexpr (kV) copy16(st + v_to + i * 512, vp + i * 512);
        }
        if (NK == 32 || (threadIdx.x & 31) < NK) {
            copy4(st + e_to, ke);
            if constexpr (kV) copy4(st + kHalf + e_to, ve);
        }
    }
    // Only the rows that exist: `left` rows from row number `lane` of the step on.
    __device__ __forceinline__ void fill_tail(uint32_t to, const uint8_t* kp, const uint8_t* vp,
                                              const uint32_t* ke, const uint32_t* ve,
                                              int left) const {
        const uint32_t st = base + to;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < NK / PASS; ++i) {
            const bool ok = lane / CH + i * PASS < left + lane;
            cp_async16(st + k_dst(i), ok ? kp + i * 512 : kp, ok);
            if constexpr (kV) cp_async16(st + v_to + i * 512, ok ? vp + i * 512 : vp, ok);
        }
        if (NK == 32 || lane < NK) {
            cp_async4(st + e_to, ke, left > 0);
            if constexpr (kV) cp_async4(st + kHalf + e_to, ve, left > 0);
        }
    }
    __device__ static __forceinline__ void copy16(uint32_t dst, const void* src) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
    }
    __device__ static __forceinline__ void copy4(uint32_t dst, const void* src) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src));
    }
    __device__ static __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
        const int n = valid ? 4 : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n));
    }

    // Bit x: slot x of the stage counts (x < NK).
    __device__ __forceinline__ uint32_t live(int s) const {
        uint32_t m;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(m) : "r"(mask_at(s)) : "memory");
        return m & (NK == 32 ? 0xffffffffu : 0xffffu);
    }

    template <int N>
    __device__ static __forceinline__ void lds(uint32_t (&w)[N], uint32_t a) {
        if constexpr (N == 1)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
        else if constexpr (N == 2)
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
        else
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(a)
                         : "memory");
    }
    // Lane's quarter of the K row in row gid of the j-th 8 rows.
    __device__ __forceinline__ void k_words(uint32_t (&w)[R::kKW], uint32_t st, int j) const {
        const uint32_t a = st + k_at + (uint32_t)(8 * j * RB);
        if constexpr (R::kKW == 8) {
            uint32_t lo[4], hi[4];
            lds<4>(lo, a);
            lds<4>(hi, st + (k_at ^ 16u) + (uint32_t)(8 * j * RB));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = lo[i];
                w[4 + i] = hi[i];
            }
        } else {
            lds<R::kKW>(w, a);
        }
    }
    // Lane's eighth of the V row of key 16 i + t + 4 je.
    __device__ __forceinline__ void v_words(uint32_t (&w)[R::kVW], uint32_t st, int i, int je) const {
        lds<R::kVW>(w, st + v_at + (uint32_t)((16 * i + 4 * je) * RB));
    }
    // Entry of row gid + 8 k of 16-key group i.
    __device__ __forceinline__ uint32_t entry(uint32_t st, int i, int k, bool v) const {
        uint32_t e[1];
        lds<1>(e, st + e_at + (v ? kHalf : 0) + 64u * i + 8u * k);
        return e[0];
    }
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    uint64_t ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 8 x 8 transpose of b16 pairs over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// ---------------------------------------------------------------- attention
// A warp's query: NH * 8 heads of a unit.  kShared: its fragments lie in shared memory
// (kBytes of it), for kernels that want the registers for a further CTA on the SM.
template <int D, int F, int NH, bool kShared = false>
struct QQuery {
    static constexpr int kBytes = kShared ? D / 16 * NH * 256 : 0;
    uint32_t qb[kShared ? 1 : NH][kShared ? 1 : D / 16][2];  // B fragments of 8 heads each
    uint32_t at = 0;                                         // this lane's, if shared
    float2 qsum[NH];  // sums of the scaled q in units of the operands, heads 8 n + 2 t, + 1
    float2 kf[NH];    // logits of the scaled q -> log2 domain

    // q: the unit's query rows, `stride` elements apart; rows from g on are zero.
    __device__ __forceinline__ void init(const __nv_bfloat16* q, size_t stride, int g,
                                         float scale_log2, uint32_t shared_at = 0) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
        at = shared_at + lane * 8;  // a lane reads what it wrote
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const int h = 8 * n + gid;
            float x[D / 4], amax = 0.f;
            const uint4* src = reinterpret_cast<const uint4*>(q + (size_t)h * stride + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = h < g ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
                    x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
            }
#pragma unroll
            for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^(14 - exponent); the exponent is held above -100, where q still fits
            const int ex = max((int)(__float_as_uint(amax) >> 23), 27) - 127;
            const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            // held in the normal range: |q| up to 2^117 at the usual scales
            const float k = fminf(fmaxf(scale_log2 / kCodeUnit<F> *
                                            __uint_as_float((uint32_t)(127 - 14 + ex) << 23), 1.2e-38f),
                                  3.4e38f);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
                x[i] *= up;
                sum += x[i];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            sum *= kCodeUnit<F>;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w = pack_f16(x[k_dim<F>(ks, 2 * e)] * odd_unit<F>(ks & 1),
                                                x[k_dim<F>(ks, 2 * e + 1)] * odd_unit<F>(ks & 1));
                    if constexpr (kShared)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + (ks * NH + n) * 256 + 4 * e),
                                     "r"(w) : "memory");
                    else qb[n][ks][e] = w;
                }
            qsum[n] = make_float2(__shfl_sync(0xffffffffu, sum, 8 * t),
                                  __shfl_sync(0xffffffffu, sum, 8 * t + 4));
            kf[n] = make_float2(__shfl_sync(0xffffffffu, k, 8 * t),
                                __shfl_sync(0xffffffffu, k, 8 * t + 4));
        }
    }

    // Logits, before kf, of the stage's keys: x[i][k][n] of row gid + 8 k of 16-key
    // group i and heads 8 n + 2 t, + 1; -inf where `live` is clear.
    template <class Ring>
    __device__ __forceinline__ void logits(float2 (&x)[Ring::NK / 16][2][NH], const Ring& ring,
                                           uint32_t st, uint32_t live) const {
        constexpr int NG = Ring::NK / 16;
        float acc[NG][NH][4];
        // groups side by side, where Q's registers are not short already
        constexpr int G = kShared ? 1 : NG;
#pragma unroll
        for (int i0 = 0; i0 < NG; i0 += G) {
            uint32_t w[G][2][Ring::R::kKW];
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i0 + i][n][e] = 0.f;
                ring.k_words(w[i][0], st, 2 * (i0 + i));
                ring.k_words(w[i][1], st, 2 * (i0 + i) + 1);
            }
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b[NH][2];
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    if constexpr (kShared) {
                        Ring::template lds<2>(b[n], at + (ks * NH + n) * 256);
                    } else {
                        b[n][0] = qb[n][ks][0];
                        b[n][1] = qb[n][ks][1];
                    }
                }
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    uint32_t a[4];
                    k_frag<F>(w[i][0], ks, a[0], a[2]);
                    k_frag<F>(w[i][1], ks, a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < NH; ++n) mma_f16(acc[i0 + i][n], a, b[n][0], b[n][1]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t ent = ring.entry(st, i, k, false);
                const float2 sc = both(entry_scale(ent)), z = both(entry_zero(ent));
#pragma unroll
                for (int n = 0; n < NH; ++n)
                    x[i][k][n] = tc::ffma2(make_float2(acc[i][n][2 * k], acc[i][n][2 * k + 1]), sc,
                                           fmul2(qsum[n], z));
            }
        }
        if (live != (Ring::NK == 32 ? 0xffffffffu : 0xffffu)) {
            const int gid = (threadIdx.x & 31) >> 2;
            const uint32_t mine = live >> ((gid >> 1) + 4 * (gid & 1));
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (!((mine >> (16 * i + 8 * k)) & 1u)) {
#pragma unroll
                        for (int n = 0; n < NH; ++n) x[i][k][n] = both(-INFINITY);
                    }
        }
    }
};

struct NoMaxima {
    template <int NG, int NH>
    __device__ __forceinline__ void operator()(int, const float2 (&)[NG][NH]) const {}
};

template <int D, int F, int NH, int kStages, bool kSharedQ = false,
          int kKeys = QRow<D, F>::kBytes <= 64 ? 32 : 16>
struct QAttend {
    using Ring = QRing<D, F, true, kStages, kKeys>;
    static constexpr int NK = Ring::NK, NG = NK / 16;

    QQuery<D, F, NH, kSharedQ> q;
    // tile m: rows dims gid D / 8 + 2 m (elements 0, 1) and + 1 (2, 3), columns heads 8 n
    // + 2 t, + 1
    float o[D / 16][NH][4];
    float2 m[NH];             // p = 2^(logit - m); m lies 10..14 below the running maximum
    float2 l[NH], zacc[NH];   // sums over the lane's keys: p, and p z with what step() moves there
    float2 off[NH];           // what recentre() took from the lane's part of O
    float up;                 // power of two above every |scale| seen: O counts in it

    __device__ __forceinline__ void init(const __nv_bfloat16* qp, size_t stride, int g,
                                         float scale_log2, uint32_t shared_q = 0) {
        q.init(qp, stride, g, scale_log2, shared_q);
        up = 0.f;
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            m[n] = both(-INFINITY);
            l[n] = zacc[n] = off[n] = both(0.f);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][n][e] = 0.f;
        }
    }

    __device__ static __forceinline__ float moved(float old, float mx, float& f) {
        const float mn = fmaxf(old, mx - 10.f);
        f = mn == -INFINITY ? 1.f : exp2f(old - mn);
        return mn;
    }
    // Moves the references to the step's maxima (log2 domain) and largest |scale|;
    // mx, sc: the lane's keys'.
    __device__ __forceinline__ void rescale(float2 (&mx)[NH], float sc) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
            sc = fmaxf(sc, __shfl_xor_sync(0xffffffffu, sc, w));
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                mx[n].x = fmaxf(mx[n].x, __shfl_xor_sync(0xffffffffu, mx[n].x, w));
                mx[n].y = fmaxf(mx[n].y, __shfl_xor_sync(0xffffffffu, mx[n].y, w));
            }
        }
        float fo = 1.f;
        if (sc > up) {
            // 2^(exponent + 1), between 2^-125 and 2^126
            const uint32_t ex = min(max(__float_as_uint(sc) >> 23, 1u) + 1u, 253u);
            const float nu = __uint_as_float(ex << 23);
            fo = up / nu;
            up = nu;
        }
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            float2 f;
            m[n].x = moved(m[n].x, mx[n].x, f.x);
            m[n].y = moved(m[n].y, mx[n].y, f.y);
            l[n] = fmul2(l[n], f);
            zacc[n] = fmul2(zacc[n], f);
            if constexpr (F == HS_KV_INT4) off[n] = fmul2(off[n], make_float2(f.x * fo, f.y * fo));
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][n][e] *= (e & 1 ? f.y : f.x) * fo;
        }
    }

    // 4-bit codes and zero points are large beside the values that they cancel to, so both
    // have to be weighted alike: the rounding of p s to fp16, the same for every key of one
    // weight and scale, would otherwise leave an offset in all dimensions (keys of equal weight
    // below a larger one: 2% of the outputs' RMS at 131072 of them, 5% at 2^20). With
    // any c0 and r = p s as rounded,
    //     sum p v^ = sum r (c - c0) + sum p (z + c0 s) + what r's rounding does to c - c0,
    // of which the last is the rounding of a weight, 2^-12 of it, where c0 is the code that
    // stands for 0.  (A c0 of 7.5 for all rows left 0.15% at 131072 one-sided values of mean 0,
    // this one 0.04%.  The sum of r c0 costs two conversions and an FMA per pair of weights:
    // 32 sequences of 131072 keys, 16 heads, 552 -> 569 us; 2048-row token layer 320 -> 334.)
    //
    // c0 for the lane's keys together: held to the codes' range (no number: 0), so that no
    // scale makes it large.
    __device__ static __forceinline__ float centre(const uint32_t (&ent)[NG][2]) {
        float s = 0.f, z = 0.f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            s += entry_scale(ent[i][0]) + entry_scale(ent[i][1]);
            z += entry_zero(ent[i][0]) + entry_zero(ent[i][1]);
        }
        return fminf(fmaxf(__fdividef(-z, s), 0.f), 15.f);
    }

    // One stage's keys.  maxima(step, .): of each 16-key group the largest logits (log2
    // domain) of the lane's two keys, heads 8 n + 2 t, + 1.
    template <class Maxima>
    __device__ __forceinline__ void step(const Ring& ring, uint32_t st, uint32_t live, int at,
                                         const Maxima& maxima) {
        float2 x[NG][2][NH];
        q.logits(x, ring, st, live);
        uint32_t ent[NG][2];
        float2 mx[NH], gm[NG][NH];
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            ent[i][0] = ring.entry(st, i, 0, true);
            ent[i][1] = ring.entry(st, i, 1, true);
            big = tc::max3f(big, fabsf(entry_scale(ent[i][0])), fabsf(entry_scale(ent[i][1])));
        }
        bool grow = big > up;
#pragma unroll
        for (int n = 0; n < NH; ++n) {
#pragma unroll
            for (int i = 0; i < NG; ++i)
                gm[i][n] = fmul2(make_float2(fmaxf(x[i][0][n].x, x[i][1][n].x),
                                             fmaxf(x[i][0][n].y, x[i][1][n].y)), q.kf[n]);
            mx[n] = gm[0][n];
            if constexpr (NG == 2)
                mx[n] = make_float2(fmaxf(mx[n].x, gm[1][n].x), fmaxf(mx[n].y, gm[1][n].y));
            grow |= mx[n].x > m[n].x + 14.f || mx[n].y > m[n].y + 14.f;
        }
        maxima(at, gm);
        if (__any_sync(0xffffffffu, grow)) rescale(mx, big);
        const float down = up == 0.f ? 0.f : __uint_as_float(0x7f000000u - __float_as_uint(up));
        const float c0 = F == HS_KV_INT4 ? centre(ent) : 0.f;
        const float2 take = both(-c0 * up);
        float2 nm[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n)
            nm[n] = make_float2(m[n].x == -INFINITY ? 0.f : -m[n].x,
                                m[n].y == -INFINITY ? 0.f : -m[n].y);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            uint32_t b[NH][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float s = entry_scale(ent[i][k]);
                float zero = entry_zero(ent[i][k]);
                if constexpr (F == HS_KV_INT4) zero = fmaf(c0, s, zero);
                const float2 z = both(zero);
                const float2 sd = both(s * down);
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    const float2 y = tc::ffma2(x[i][k][n], q.kf[n], nm[n]);
                    const float2 p = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                    l[n] = tc::fadd2(l[n], p);
                    zacc[n] = tc::ffma2(p, z, zacc[n]);
                    const float2 w = fmul2(p, sd);
                    const __half2 r = __floats2half2_rn(w.x, w.y);
                    if constexpr (F == HS_KV_INT4)
                        zacc[n] = tc::ffma2(__half22float2(r), take, zacc[n]);
                    b[n][k] = transpose8(*reinterpret_cast<const uint32_t*>(&r));
                }
            }
            uint32_t v[4][Ring::R::kVW];
#pragma unroll
            for (int je = 0; je < 4; ++je) ring.v_words(v[je], st, i, je);
#pragma unroll
            for (int j = 0; j < D / 8; j += 4) {
                uint32_t p0[4], p1[4];
                v_pairs<F>(v[0], v[1], j, p0);
                v_pairs<F>(v[2], v[3], j, p1);
                const uint32_t a0[4] = {p0[0], p0[1], p1[0], p1[1]};
                const uint32_t a1[4] = {p0[2], p0[3], p1[2], p1[3]};
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    mma_f16(o[j / 2][n], a0, b[n][0], b[n][1]);
                    mma_f16(o[j / 2 + 1][n], a1, b[n][0], b[n][1]);
                }
            }
        }
    }

    // The matrix unit cuts sums off where they lose bits, and 4-bit codes are positive: O
    // would carry the codes' mean, up to many times what is left of it once the zero points
    // are in, and lose a little of it each time (131072 keys of equal weight, 886 sums a warp:
    // outputs 3.1% of their RMS too low).  So every kRecentre steps each head's mean over
    // the lane's dimensions moves into an fp32 sum of its own (0.2%, the outputs' rounding,
    // at 8, 16 and 32 steps, which cost 21, 16 and 13 of 536 us).
    static constexpr int kRecentre = 16;
    __device__ __forceinline__ void recentre() {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            float2 s = both(0.f);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                s = tc::ffma2(make_float2(o[j][n][2], o[j][n][3]), both(odd_unit<F>(1)),
                              tc::fadd2(s, make_float2(o[j][n][0], o[j][n][1])));
            const float2 a = fmul2(s, both(1.f / (D / 8)));
            off[n] = tc::fadd2(off[n], a);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[j][n][e] = fmaf(e & 1 ? a.y : a.x, -1.f / odd_unit<F>(e >> 1), o[j][n][e]);
        }
    }
    // To be called after the i-th step (from 0) of a run.
    __device__ __forceinline__ void stepped(int i) {
        if constexpr (F == HS_KV_INT4)
            if (i % kRecentre == kRecentre - 1) recentre();
    }

    // Steps first, first + stride, ... below n_steps of a source's list.
    template <class Src, class Maxima>
    __device__ __forceinline__ void run(const Ring& ring, const QuantCache& c, const Src& src,
                                        int first, int stride, int n_steps, const Maxima& maxima) {
        // copies run kStages - 1 steps ahead, the keys' places one more, index entries two
        int ahead = first;
        QPlace at = find<NK>(src, src.load(first), first, n_steps);
        int word = first + stride < n_steps ? src.load(first + stride) : 0;
        auto fill = [&](int s) {
            if (ahead < n_steps) ring.fill(s, c, row_of(src.pm, at), at.run);
            cp_async_commit();
            ahead += stride;
            at = find<NK>(src, word, ahead, n_steps);
            if (ahead + stride < n_steps) word = src.load(ahead + stride);
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fill(i);
        int s = 0, fs = kStages - 1, done = 0;
        for (int st = first; st < n_steps; st += stride) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            fill(fs);
            step(ring, ring.stage(s), ring.live(s), st, maxima);
            stepped(done++);
            s = s + 1 == kStages ? 0 : s + 1;
            fs = fs + 1 == kStages ? 0 : fs + 1;
        }
        cp_async_wait<0>();
        __syncwarp();  // the ring may be reused
    }

    // The same for rows 0 .. n - 1 of the bases, kStride steps apart: running pointers in
    // place of row numbers (a hundred cycles of 1400 a step, at 16 heads of 128).
    template <int kStride, class Maxima>
    __device__ __forceinline__ void run_dense(const Ring& ring, const QuantCache& c, int n,
                                              int first, int n_steps, const Maxima& maxima) {
        const int lane = threadIdx.x & 31;
        constexpr uint32_t kRow = kStride * NK, kEnd = kStages * Ring::kStage;
        const size_t r0 = (size_t)first * NK;
        const uint8_t* kp = c.kc + r0 * Ring::RB + lane * 16;
        const uint8_t* vp = c.vc + r0 * Ring::RB + lane * 16;
        const uint32_t *ke = c.ks + r0 + lane, *ve = c.vs + r0 + lane;
        int ahead = first;
        uint32_t to = 0, at = 0;  // stages' offsets: filled next, read next
        auto fill = [&] {
            if (ahead < n_steps) {
                const int left = n - ahead * NK - lane;  // keys from the lane's on
                if ((ahead + 1) * NK <= n) ring.fill_dense(to, kp, vp, ke, ve);
                else ring.fill_tail(to, kp, vp, ke, ve, left);
                kp += kRow * Ring::RB;
                vp += kRow * Ring::RB;
                ke += kRow;
                ve += kRow;
            }
            cp_async_commit();
            ahead += kStride;
            to = to + Ring::kStage == kEnd ? 0u : to + Ring::kStage;
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fill();
        for (int st = first; st < n_steps; st += kStride) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            fill();
            const int left = n - st * NK;
            const uint32_t live = left >= NK ? (NK == 32 ? 0xffffffffu : 0xffffu) : (1u << left) - 1u;
            step(ring, ring.base + at, live, st, maxima);
            stepped((st - first) / kStride);
            at = at + Ring::kStage == kEnd ? 0u : at + Ring::kStage;
        }
        cp_async_wait<0>();
        __syncwarp();
    }

    // Sums over the warp, puts O in its own units and adds the zero points:
    // o = sum p v^, l = sum p.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            // what the lane's dimensions have in common
            float2 base;
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) {
                l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, w);
                l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, w);
                zacc[n].x += __shfl_xor_sync(0xffffffffu, zacc[n].x, w);
                zacc[n].y += __shfl_xor_sync(0xffffffffu, zacc[n].y, w);
            }
            base.x = fmaf(off[n].x * (1.f / kCodeUnit<F>), up, zacc[n].x);
            base.y = fmaf(off[n].y * (1.f / kCodeUnit<F>), up, zacc[n].y);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[j][n][e] = fmaf(o[j][n][e] * (odd_unit<F>(e >> 1) / kCodeUnit<F>), up,
                                      e & 1 ? base.y : base.x);
        }
    }

    // After finish, of head 8 n + 2 t + e: the lane's D / 8 dimensions from gid D / 8 on.
    __device__ __forceinline__ float dim(int n, int e, int x) const { return o[x >> 1][n][2 * (x & 1) + e]; }
    static constexpr int kPart = 32 + 16 * D;  // floats of a partial

    // Partial: part[2 h] = m, part[2 h + 1] = l, then O rows of D floats at part + 32
    // (16 heads).
    __device__ __forceinline__ void store_part(float* part, int g) const {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * n + 2 * t + e;
                if (h >= g) continue;
                if (gid == 0) {
                    part[2 * h] = e ? m[n].y : m[n].x;
                    part[2 * h + 1] = e ? l[n].y : l[n].x;
                }
                float* row = part + 32 + h * D + gid * (D / 8);
#pragma unroll
                for (int x = 0; x < D / 8; x += 4)
                    *reinterpret_cast<float4*>(row + x) = make_float4(
                        dim(n, e, x), dim(n, e, x + 1), dim(n, e, x + 2), dim(n, e, x + 3));
            }
    }
};

// Bases of unit (b, u): a contiguous cache's rows of that unit, or the pool.
template <int D, int F>
__device__ __forceinline__ QuantCache unit_cache(const KParams& p, const QuantCache& c, int unit) {
    if (p.bt) return c;
    const size_t r0 = (size_t)unit * p.t_kv;
    constexpr int RB = QRow<D, F>::kBytes;
    return QuantCache{c.kc + r0 * RB, c.ks + r0, c.vc + r0 * RB, c.vs + r0};
}

}  // namespace hs

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
// instructions: a 4-bit code in a byte, read as e4m3, is the number c 2^-9,
// exactly, for all of 0..15 (subnormals, then the first binade), so both formats use
// the conversion of e4m3 pairs.  What fp16's range needs:
//  - q is scaled by a power of two per head so that max|q| lies in [2^14, 2^15);
//    a bf16 element is then exact unless it is 2^-29 of the largest or less
//    (error 2^-39 of the largest);
//  - p_i s_i is taken relative to 2^10 at the running maximum (growing to
//    2^14 before O is rescaled) and to a power of two above the largest |s_i|
//    seen, and rounded to fp16: relative 2^-12 for weights down to 2^-24 of the
//    largest, an absolute 2^-35 of it below.
// Everything else is fp32.  What bounds the kernels is the issue rate: mma.sync
// holds its scheduler for 8 cycles (measured alone 8.7 cycles, with 4 FFMAs beside it
// 12.8, with 8 of them 17), so 16 keys of 128 dims take 256 issue cycles for their
// 32 MMAs beside some 250 for unpacking, the softmax and the reads.
//
// One warp, 16 heads as the rows of mma.m16n8k16, 16 keys at a time.  Lane
// (gid, t) of the warp (gid = lane / 4, t = lane % 4) needs of a key's K row the
// t-th quarter and of a V row the gid-th eighth (Q's fragments take the same
// order of dimensions), so rows are read from shared memory as they lie in the
// cache.  cp.async fills a ring of stages per warp; it also places the rows:
// within 16 keys, key t + 4 e + 8 j is column 2 t + e of 8-column tile j, K rows lie in
// column order, V rows keep their order with 16-byte chunks swizzled, a lane's
// four entries are adjacent: every shared read is free of bank conflicts.
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

// What a code of 1 counts for in the operands.
template <int F> constexpr float kCodeUnit = F == HS_KV_INT4 ? 1.f / 512.f : 1.f;

// Dimension (of a quarter row) that element e (0: b0 low, 1: b0 high, 2: b1
// low, 3: b1 high) of k step `ks` holds.
template <int F>
__host__ __device__ constexpr int k_dim(int ks, int e) {
    return F == HS_KV_INT4 ? 8 * (ks >> 1) + (ks & 1) + 2 * e : 4 * ks + e;
}

// B fragment (b0, b1) of k step `ks` from a lane's quarter of a K row.
template <int F, int N>
__device__ __forceinline__ void k_frag(const uint32_t (&w)[N], int ks, uint32_t& b0, uint32_t& b1) {
    if constexpr (F == HS_KV_INT4)
        e4m3_f16((ks & 1 ? w[ks >> 1] >> 4 : w[ks >> 1]) & 0x0f0f0f0fu, b0, b1);
    else
        e4m3_f16(w[ks], b0, b1);
}

// Pairs (a[j + i], b[j + i]), i = 0..3, of a lane's eighths of two V rows, j a
// multiple of 4.
template <int F, int N>
__device__ __forceinline__ void v_pairs(const uint32_t (&a)[N], const uint32_t (&b)[N], int j,
                                        uint32_t (&p)[4]) {
    if constexpr (F == HS_KV_INT4) {
        // bytes (a, b, a, b) of two neighbouring bytes of each row
        const uint32_t x = __byte_perm(a[j >> 3], b[j >> 3], (j & 4) ? 0x7362 : 0x5140);
        e4m3_f16(x & 0x0f0f0f0fu, p[0], p[2]);
        e4m3_f16((x >> 4) & 0x0f0f0f0fu, p[1], p[3]);
    } else {
        e4m3_f16(__byte_perm(a[j >> 2], b[j >> 2], 0x5140), p[0], p[1]);
        e4m3_f16(__byte_perm(a[j >> 2], b[j >> 2], 0x7362), p[2], p[3]);
    }
}

// ------------------------------------------------------------- row sources
// row(slot) = row, relative to the bases handed to the warp, of key slot
// 0..n-1 of its list, -1 if that slot is masked or out of range.

// Consecutive rows first + slot of a contiguous cache.
struct QRange {
    static constexpr bool kDirect = true;  // cheap: each lane asks for what it loads
    int first, n;
    __device__ __forceinline__ int row(int slot) const { return slot < n ? first + slot : -1; }
};
// Logical keys first + slot through the block table.
struct QPagedRange {
    static constexpr bool kDirect = false;
    int first, n;
    PageMap pm;
    __device__ __forceinline__ int row(int slot) const {
        return slot < n ? pm.row(first + slot) : -1;
    }
};
// Entries of an index row (token mode: keys; block mode: blocks clipped to
// keys <= t), through the block table if there is one.
struct QIndex {
    static constexpr bool kDirect = false;
    const int32_t* ids;
    int n, B, t;
    bool paged;
    PageMap pm;
    __device__ __forceinline__ int row(int slot) const {
        if (slot >= n) return -1;
        int key;
        if (B == 1) {
            key = __ldg(ids + slot);
            if (key < 0 || key > t) { set_status(HS_ERR_BOUNDS); return -1; }
        } else {
            const int jb = slot / B;
            const int id = __ldg(ids + jb);
            if (id < 0 || id > t / B) { set_status(HS_ERR_BOUNDS); return -1; }
            key = id * B + (slot - jb * B);
            if (key > t) return -1;
        }
        return paged ? pm.row(key) : key;
    }
};

// -------------------------------------------------------------- ring of rows
// A warp's stages.  K only: the V half is neither filled nor reserved.
template <int D, int F, bool kV, int kStages>
struct QRing {
    using R = QRow<D, F>;
    static constexpr int RB = R::kBytes;
    static constexpr int NK = RB <= 64 ? 32 : 16;        // keys of a stage
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
        e_at = (uint32_t)(kKeyBytes + 16 * t);
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

    // Starts the copies of the step whose first slot is slot0.  `mine`: row of
    // slot slot0 + lane % NK, for sources that are not direct.
    template <class Src>
    __device__ __forceinline__ void fill(int s, const QuantCache& c, const Src& src, int slot0,
                                         int mine) const {
        const int lane = threadIdx.x & 31;
        const uint32_t st = stage(s);
        if constexpr (Src::kDirect) {
            const int r0 = src.first + slot0;
            if (slot0 + NK <= src.n) {  // a whole step: consecutive bytes
                const uint8_t* kp = c.kc + (size_t)r0 * RB + lane * 16;
                const uint8_t* vp = c.vc + (size_t)r0 * RB + lane * 16;
#pragma unroll
                for (int i = 0; i < NK / PASS; ++i) {
                    copy16(st + k_dst(i), kp + i * 512);
                    if constexpr (kV) copy16(st + v_to + i * 512, vp + i * 512);
                }
                if (NK == 32 || lane < NK) {
                    copy4(st + e_to, c.ks + (size_t)r0 + lane);
                    if constexpr (kV) copy4(st + kHalf + e_to, c.vs + (size_t)r0 + lane);
                }
                return;
            }
            mine = src.row(slot0 + (lane & (NK - 1)));
        }
        const uint32_t live = __ballot_sync(0xffffffffu, mine >= 0);
        if (live == 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < NK / PASS; ++i) {
                const uint32_t r = __shfl_sync(0xffffffffu, mine, lane / CH + i * PASS);
                const size_t off = (size_t)r * RB + (lane % CH) * 16;
                copy16(st + k_dst(i), c.kc + off);
                if constexpr (kV) copy16(st + v_to + i * 512, c.vc + off);
            }
            if (NK == 32 || lane < NK) {
                copy4(st + e_to, c.ks + (uint32_t)mine);
                if constexpr (kV) copy4(st + kHalf + e_to, c.vs + (uint32_t)mine);
            }
        } else {  // rows that do not count are zeros
#pragma unroll
            for (int i = 0; i < NK / PASS; ++i) {
                const int r = __shfl_sync(0xffffffffu, mine, lane / CH + i * PASS);
                const size_t off = r >= 0 ? (size_t)r * RB + (lane % CH) * 16 : 0;
                cp_async16(st + k_dst(i), c.kc + off, r >= 0);
                if constexpr (kV) cp_async16(st + v_to + i * 512, c.vc + off, r >= 0);
            }
            if (NK == 32 || lane < NK) {
                const size_t off = mine >= 0 ? (size_t)mine : 0;
                cp_async4(st + e_to, c.ks + off, mine >= 0);
                if constexpr (kV) cp_async4(st + kHalf + e_to, c.vs + off, mine >= 0);
            }
        }
        if constexpr (!Src::kDirect) {
            if (lane == 0)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(mask_at(s)), "r"(live) : "memory");
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

    // Bit x: slot slot0 + x counts (x < NK).
    template <class Src>
    __device__ __forceinline__ uint32_t live(int s, const Src& src, int slot0) const {
        constexpr uint32_t kAll = NK == 32 ? 0xffffffffu : 0xffffu;
        if constexpr (Src::kDirect) {
            const int left = src.n - slot0;
            return left >= NK ? kAll : (1u << max(left, 0)) - 1u;
        } else {
            uint32_t m;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(m) : "r"(mask_at(s)) : "memory");
            return m & kAll;
        }
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
    // Lane's quarter of the K row in column gid of tile j.
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
    // Entries of keys t, t + 4, t + 8, t + 12 of 16-key group i.
    __device__ __forceinline__ void entries(uint32_t (&e)[4], uint32_t st, int i, bool v) const {
        lds<4>(e, st + e_at + (v ? kHalf : 0) + 64u * i);
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

// Scales and zero points of two entries.
__device__ __forceinline__ void entry_pair(uint32_t e0, uint32_t e1, float2& sc, float2& z) {
    sc = make_float2(entry_scale(e0), entry_scale(e1));
    z = make_float2(entry_zero(e0), entry_zero(e1));
}

// ---------------------------------------------------------------- attention
// A warp's query: 16 heads of a unit.
template <int D, int F>
struct QQuery {
    uint32_t qf[D / 16][4];
    float qsum[2];  // sum of the scaled q in units of the operands, heads gid and gid + 8
    float kf[2];    // logit of the scaled q -> log2 domain

    // q: the unit's query rows, `stride` elements apart; rows g..15 are zero.
    __device__ __forceinline__ void init(const __nv_bfloat16* q, size_t stride, int g,
                                         float scale_log2) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const bool ok = gid + 8 * hr < g;
            float x[D / 4], amax = 0.f;
            const uint4* src =
                reinterpret_cast<const uint4*>(q + (size_t)(gid + 8 * hr) * stride + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = ok ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
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
            kf[hr] = fmaxf(scale_log2 / kCodeUnit<F> *
                               __uint_as_float((uint32_t)(127 - 14 + ex) << 23), 1.2e-38f);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
                x[i] *= up;
                sum += x[i];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qsum[hr] = sum * kCodeUnit<F>;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qf[ks][2 * e + hr] = pack_f16(x[k_dim<F>(ks, 2 * e)], x[k_dim<F>(ks, 2 * e + 1)]);
        }
    }

    // Logits, before kf, of the stage's keys: x[j][hr] of keys t + 8 j (.x) and t + 4
    // + 8 j (.y) past each 16 (j even: the first 8 of them) and head gid + 8 hr; -inf
    // where `live` is clear.
    template <class Ring>
    __device__ __forceinline__ void logits(float2 (&x)[Ring::NK / 8][2], const Ring& ring,
                                           uint32_t st, uint32_t live) const {
        constexpr int NT = Ring::NK / 8;
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
            uint32_t w[Ring::R::kKW];
            ring.k_words(w, st, j);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b0, b1;
                k_frag<F>(w, ks, b0, b1);
                mma_f16(acc[j], qf[ks], b0, b1);
            }
        }
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            uint32_t ent[4];
            ring.entries(ent, st, i, false);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                float2 sc, z;
                entry_pair(ent[2 * jj], ent[2 * jj + 1], sc, z);
                const float* a = acc[2 * i + jj];
#pragma unroll
                for (int hr = 0; hr < 2; ++hr)
                    x[2 * i + jj][hr] = tc::ffma2(make_float2(a[2 * hr], a[2 * hr + 1]), sc,
                                                  fmul2(both(qsum[hr]), z));
            }
        }
        if (live != (Ring::NK == 32 ? 0xffffffffu : 0xffffu)) {
            const uint32_t mine = live >> (threadIdx.x & 3);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (!((mine >> (8 * j)) & 1u)) x[j][0].x = x[j][1].x = -INFINITY;
                if (!((mine >> (8 * j + 4)) & 1u)) x[j][0].y = x[j][1].y = -INFINITY;
            }
        }
    }
};

struct NoMaxima {
    __device__ __forceinline__ void operator()(int, float, float) const {}
};

template <int D, int F, int kStages>
struct QAttend {
    using Ring = QRing<D, F, true, kStages>;
    static constexpr int NK = Ring::NK, NT = NK / 8;

    QQuery<D, F> q;
    float o[D / 8][4];  // tile j, element e: head gid + 8 (e / 2), dim (2t + e % 2) D / 8 + j
    float m[2];         // p = 2^(logit - m); m lies 10..14 below the running maximum
    float2 l[2], zacc[2];       // sums of p and p z' (two shares a lane, a lane's keys)
    float up;                   // power of two above every |scale| seen: O counts in it

    __device__ __forceinline__ void init(const __nv_bfloat16* qp, size_t stride, int g,
                                         float scale_log2) {
        q.init(qp, stride, g, scale_log2);
        up = 0.f;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            m[hr] = -INFINITY;
            l[hr] = zacc[hr] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }

    // Moves the references to the step's maxima (log2 domain) and largest |scale|.
    __device__ __forceinline__ void rescale(float mx0, float mx1, float sc) {
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) sc = fmaxf(sc, __shfl_xor_sync(0xffffffffu, sc, w));
        float fo = 1.f;
        if (sc > up) {
            // 2^(exponent + 1), between 2^-125 and 2^126
            const uint32_t ex = min(max(__float_as_uint(sc) >> 23, 1u) + 1u, 253u);
            const float nu = __uint_as_float(ex << 23);
            fo = up / nu;
            up = nu;
        }
        const float mx[2] = {mx0, mx1};
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const float mn = fmaxf(m[hr], mx[hr] - 10.f);
            const float f = mn == -INFINITY ? 1.f : exp2f(m[hr] - mn);
            m[hr] = mn;
            l[hr] = fmul2(l[hr], both(f));
            zacc[hr] = fmul2(zacc[hr], both(f));
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][2 * hr] *= f * fo;
                o[j][2 * hr + 1] *= f * fo;
            }
        }
    }

    // One stage's keys.  maxima(step, head gid's, head gid + 8's): the step's
    // largest logit per head, log2 domain, the same in a quad.
    template <class Maxima>
    __device__ __forceinline__ void step(const Ring& ring, uint32_t st, uint32_t live, int at,
                                         const Maxima& maxima) {
        float2 x[NT][2];
        q.logits(x, ring, st, live);
        uint32_t ent[NT / 2][4];
        float mx[2], big = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            ring.entries(ent[i], st, i, true);
#pragma unroll
            for (int je = 0; je < 4; je += 2)
                big = tc::max3f(big, fabsf(entry_scale(ent[i][je])), fabsf(entry_scale(ent[i][je + 1])));
        }
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            mx[hr] = fmaxf(x[0][hr].x, x[0][hr].y);
#pragma unroll
            for (int j = 1; j < NT; ++j) mx[hr] = tc::max3f(mx[hr], x[j][hr].x, x[j][hr].y);
            mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 1));
            mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 2));
            mx[hr] *= q.kf[hr];
        }
        maxima(at, mx[0], mx[1]);
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 14.f || mx[1] > m[1] + 14.f || big > up))
            rescale(mx[0], mx[1], big);
        const float down = up == 0.f ? 0.f : __uint_as_float(0x7f000000u - __float_as_uint(up));
        const float nm[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            uint32_t a[4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                float2 sc, z;
                entry_pair(ent[i][2 * jj], ent[i][2 * jj + 1], sc, z);
                sc = fmul2(sc, both(down));
#pragma unroll
                for (int hr = 0; hr < 2; ++hr) {
                    const float2 y = tc::ffma2(x[2 * i + jj][hr], both(q.kf[hr]), both(nm[hr]));
                    const float2 p = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                    l[hr] = tc::fadd2(l[hr], p);
                    zacc[hr] = tc::ffma2(p, z, zacc[hr]);
                    const float2 w = fmul2(p, sc);
                    a[2 * jj + hr] = pack_f16(w.x, w.y);
                }
            }
            uint32_t v[4][Ring::R::kVW];
#pragma unroll
            for (int je = 0; je < 4; ++je) ring.v_words(v[je], st, i, je);
#pragma unroll
            for (int j = 0; j < D / 8; j += 4) {
                uint32_t b0[4], b1[4];
                v_pairs<F>(v[0], v[1], j, b0);
                v_pairs<F>(v[2], v[3], j, b1);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_f16(o[j + e], a, b0[e], b1[e]);
            }
        }
    }

    // Steps first, first + stride, ... below n_steps of a source's list.
    template <class Src, class Maxima>
    __device__ __forceinline__ void run(const Ring& ring, const QuantCache& c, const Src& src,
                                        int first, int stride, int n_steps, const Maxima& maxima) {
        const int lane = threadIdx.x & 31;
        auto mine = [&](int st) {
            if constexpr (Src::kDirect) return 0;
            else return st < n_steps ? src.row(st * NK + (lane & (NK - 1))) : -1;
        };
        // copies run kStages - 1 steps ahead, the rows' places one more
        int ahead = first;
        int row = mine(first);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (ahead < n_steps) ring.fill(i, c, src, ahead * NK, row);
            cp_async_commit();
            ahead += stride;
            row = mine(ahead);
        }
        int s = 0, fs = kStages - 1;
        for (int st = first; st < n_steps; st += stride) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            if (ahead < n_steps) ring.fill(fs, c, src, ahead * NK, row);
            cp_async_commit();
            ahead += stride;
            row = mine(ahead);
            step(ring, ring.stage(s), ring.live(s, src, st * NK), st, maxima);
            s = s + 1 == kStages ? 0 : s + 1;
            fs = fs + 1 == kStages ? 0 : fs + 1;
        }
        cp_async_wait<0>();
        __syncwarp();  // the ring may be reused
    }

    // Sums over the quad, puts O in its own units and adds the zero points:
    // o = sum p v^, l[hr].x = sum p.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            float s = l[hr].x + l[hr].y, z = zacc[hr].x + zacc[hr].y;
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            l[hr].x = s;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][2 * hr] = fmaf(o[j][2 * hr], up / kCodeUnit<F>, z);
                o[j][2 * hr + 1] = fmaf(o[j][2 * hr + 1], up / kCodeUnit<F>, z);
            }
        }
    }

    // Partial (after finish): part[2 h] = m, part[2 h + 1] = l, then O rows of D
    // floats at part + 32 (16 heads).
    __device__ __forceinline__ void store_part(float* part, int g) const {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const int h = gid + 8 * hr;
            if (h >= g) continue;
            if (t == 0) {
                part[2 * h] = m[hr];
                part[2 * h + 1] = l[hr].x;
            }
            float* row = part + 32 + h * D + t * (D / 4);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < D / 8; j += 4)
                    *reinterpret_cast<float4*>(row + e * (D / 8) + j) =
                        make_float4(o[j][2 * hr + e], o[j + 1][2 * hr + e], o[j + 2][2 * hr + e],
                                    o[j + 3][2 * hr + e]);
        }
    }
    static constexpr int kPart = 32 + 16 * D;  // floats of a partial
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

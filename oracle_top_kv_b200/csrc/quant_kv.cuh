// quant_kv.cuh -- rows of a quantised K^F/V^F cache: their storage, and
// attention over them with the codes as matrix operands.
//
// A stored row is head_dim codes plus one 4-byte entry {scale, zero} (bf16
// each); code c stands for scale * c + zero.  HS_KV_INT4: c = 0..15, element
// 2j in the low and 2j + 1 in the high nibble of byte j.  HS_KV_FP8: c is an
// e4m3 number, one byte per element.
//
// Attention never rebuilds the values.  For a key with entry (s, z),
//     scale q.k^ = tau (s (q.c') + z' sum(q)),
//     sum_i p_i v^_i = sum_i (p_i s_i) c'_i + sum_i p_i z'_i,
// with c' = c - 8, z' = z + 8 s in 4 bits and c' = c, z' = z in 8.  c' is exact in
// bf16, so both products run on codes, and scale and zero are applied to the
// logits, to P and to one running sum per head: two roundings fewer than with
// rows rebuilt in bf16 first, and no multiply per element.  p_i s_i is rounded
// to bf16 for its product (relative 2^-9, as the bf16 kernels round p_i);
// everything else is fp32.
//
// One warp, 16 heads as the rows of mma.m16n8k16.  Lane (gid, t) of the warp
// (gid = lane / 4, t = lane % 4) reads straight from the cache what its
// fragments need, with no pass through shared memory: of key gid of an 8-key
// tile the t-th quarter of the row (Q's fragments take the same order of
// dimensions), and of the V rows of keys 2t and 2t + 1 the gid-th eighth.
#pragma once

#include "attend_mma.cuh"
#include "hs_common.cuh"
#include "hs_kernels.cuh"

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

template <int N>
__device__ __forceinline__ void ldg_words(uint32_t (&w)[N], const uint8_t* p, bool ok) {
    if (!ok) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0u;
        return;
    }
    if constexpr (N == 1) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (N == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ float entry_scale(uint32_t e) { return __uint_as_float(e << 16); }
__device__ __forceinline__ float entry_zero(uint32_t e) { return __uint_as_float(e & 0xffff0000u); }

__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                     *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Two 4-bit codes, in the low nibbles of x's halves, as bf16 pair c - 8:
// 0x4300 | c is the bf16 number 128 + c, and the subtraction is exact.
__device__ __forceinline__ uint32_t int4_pair(uint32_t x) {
    return bf2_sub((x & 0x000f000fu) | 0x43004300u, 0x43084308u);
}
// Two e4m3 codes, in the high bytes of x's halves, as a bf16 pair: sign, exponent
// and mantissa moved to bf16's places give the number times 2^-120 (subnormals
// too), and the product with 2^120 is exact.
__device__ __forceinline__ uint32_t fp8_pair(uint32_t x) {
    return bf2_mul(((x >> 4) & 0x07f007f0u) | (x & 0x80008000u), 0x7b807b80u);
}

// Dimension (of a quarter row) that element e (0: b0 low, 1: b0 high, 2: b1
// low, 3: b1 high) of k step `ks` holds.
template <int F>
__host__ __device__ constexpr int k_dim(int ks, int e) {
    return F == HS_KV_INT4 ? 8 * (ks >> 1) + 2 * (ks & 1) + (e >> 1) + 4 * (e & 1)
                           : 4 * ks + (e >> 1) + 2 * (e & 1);
}

// B fragment (b0, b1) of k step `ks` from a lane's quarter of a K row.
template <int F, int N>
__device__ __forceinline__ void k_frag(const uint32_t (&w)[N], int ks, uint32_t& b0, uint32_t& b1) {
    if constexpr (F == HS_KV_INT4) {
        const uint32_t x = w[ks >> 1] >> (8 * (ks & 1));
        b0 = int4_pair(x);
        b1 = int4_pair(x >> 4);
    } else {
        b0 = fp8_pair(w[ks] << 8);
        b1 = fp8_pair(w[ks]);
    }
}

// The pair (a[j], b[j]) of element j of two lanes' eighths of V rows.
template <int F, int N>
__device__ __forceinline__ uint32_t v_pair(const uint32_t (&a)[N], const uint32_t (&b)[N], int j) {
    if constexpr (F == HS_KV_INT4) {
        const uint32_t x = __byte_perm(a[j >> 3], b[j >> 3], (j & 4) ? 0x7632 : 0x5410);
        return int4_pair(x >> (4 * (j & 3)));
    } else {
        const int i = j & 3;  // bytes (any, a_i, any, b_i)
        return fp8_pair(__byte_perm(a[j >> 2], b[j >> 2], (i << 4) | ((4 + i) << 12)));
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

// ---------------------------------------------------------------- attention
// NK: keys of one step of a warp (16 or 32).
template <int D, int F, int NK>
struct QAttend {
    using R = QRow<D, F>;
    static constexpr int NT = NK / 8;  // 8-key tiles

    uint32_t qf[D / 16][4];
    float qsum[2];       // sum of q, heads gid and gid + 8
    float o[D / 8][4];   // tile j, element e: head gid + 8 (e / 2), dim (2t + e % 2) D / 8 + j
    float m[2], l[2], zacc[2];

    struct Regs {
        uint32_t k[NT][R::kKW], v[NT][2][R::kVW], ks[NT][2], vs[NT][2];
        uint32_t live;  // bit 2j + e: key 8j + 2t + e counts
    };

    // q: the unit's query rows, `stride` elements apart; rows g..15 are zero.
    __device__ __forceinline__ void init(const __nv_bfloat16* q, size_t stride, int g) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
        qsum[0] = qsum[1] = 0.f;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const bool ok = gid + 8 * hr < g;
            __nv_bfloat16 x[D / 4];
            const uint4* src =
                reinterpret_cast<const uint4*>(q + (size_t)(gid + 8 * hr) * stride + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                reinterpret_cast<uint4*>(x)[i] = ok ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < D / 4; ++i) qsum[hr] += __bfloat162float(x[i]);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __nv_bfloat162 pr =
                        __halves2bfloat162(x[k_dim<F>(ks, 2 * e)], x[k_dim<F>(ks, 2 * e + 1)]);
                    qf[ks][2 * e + hr] = *reinterpret_cast<const uint32_t*>(&pr);
                }
            }
            qsum[hr] += __shfl_xor_sync(0xffffffffu, qsum[hr], 1);
            qsum[hr] += __shfl_xor_sync(0xffffffffu, qsum[hr], 2);
            m[hr] = -INFINITY;
            l[hr] = zacc[hr] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }

    // Issues the loads of one step.  `mine`: row of slot (step's first + lane),
    // for sources that are not direct.
    template <class Src>
    __device__ __forceinline__ static void load(Regs& r, const QuantCache& c, const Src& src,
                                                int slot0, int mine) {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
        auto row = [&](int x) {
            if constexpr (Src::kDirect) return src.row(slot0 + x);
            else return __shfl_sync(0xffffffffu, mine, x);
        };
        r.live = 0u;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int rk = row(8 * j + gid);
            ldg_words<R::kKW>(r.k[j], c.kc + (size_t)rk * R::kBytes + t * (R::kBytes / 4), rk >= 0);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rv = row(8 * j + 2 * t + e);
                r.ks[j][e] = rv >= 0 ? __ldg(c.ks + rv) : 0u;
                r.vs[j][e] = rv >= 0 ? __ldg(c.vs + rv) : 0u;
                ldg_words<R::kVW>(r.v[j][e], c.vc + (size_t)rv * R::kBytes + gid * (R::kBytes / 8),
                                  rv >= 0);
                if (rv >= 0) r.live |= 1u << (2 * j + e);
            }
        }
    }

    __device__ __forceinline__ void step(const Regs& r, float scale_log2) {
        float s[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b0, b1;
                k_frag<F>(r.k[j], ks, b0, b1);
                mma_bf16(s[j], qf[ks], b0, b1);
            }
        }
        // logits in the log2 domain; masked keys -inf
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float sc = entry_scale(r.ks[j][e]);
                float z = entry_zero(r.ks[j][e]);
                if constexpr (F == HS_KV_INT4) z = fmaf(8.f, sc, z);
                const float s2 = sc * scale_log2, z2 = z * scale_log2;
                const bool ok = (r.live >> (2 * j + e)) & 1u;
#pragma unroll
                for (int hr = 0; hr < 2; ++hr) {
                    float& x = s[j][2 * hr + e];
                    x = ok ? fmaf(x, s2, qsum[hr] * z2) : -INFINITY;
                    mx[hr] = fmaxf(mx[hr], x);
                }
            }
        }
        // the reference may lag the maximum by up to 2^8 before O is rescaled
        bool grow = false;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 1));
            mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 2));
            grow |= mx[hr] > m[hr] + 8.f;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
                const float mn = fmaxf(m[hr], mx[hr]);
                const float f = mn == -INFINITY ? 1.f : exp2f(m[hr] - mn);
                m[hr] = mn;
                l[hr] *= f;
                zacc[hr] *= f;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][2 * hr] *= f;
                    o[j][2 * hr + 1] *= f;
                }
            }
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            uint32_t a[4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int j = 2 * i + jj;
                float w[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float sc = entry_scale(r.vs[j][e]);
                    float z = entry_zero(r.vs[j][e]);
                    if constexpr (F == HS_KV_INT4) z = fmaf(8.f, sc, z);
#pragma unroll
                    for (int hr = 0; hr < 2; ++hr) {
                        const float p = exp2f(s[j][2 * hr + e] - mu[hr]);
                        l[hr] += p;
                        zacc[hr] = fmaf(p, z, zacc[hr]);
                        w[2 * hr + e] = p * sc;
                    }
                }
                a[2 * jj] = pack_bf16(w[0], w[1]);
                a[2 * jj + 1] = pack_bf16(w[2], w[3]);
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                const uint32_t b0 = v_pair<F>(r.v[2 * i][0], r.v[2 * i][1], j);
                const uint32_t b1 = v_pair<F>(r.v[2 * i + 1][0], r.v[2 * i + 1][1], j);
                mma_bf16(o[j], a, b0, b1);
            }
        }
    }

    // Steps first, first + stride, ... below n_steps of a source's list.
    template <class Src>
    __device__ __forceinline__ void run(const QuantCache& c, const Src& src, int first, int stride,
                                        int n_steps, float scale_log2) {
        if (first >= n_steps) return;
        const int lane = threadIdx.x & 31;
        auto mine = [&](int st) {
            if constexpr (Src::kDirect) return 0;
            else return st < n_steps ? src.row(st * NK + (lane & (NK - 1))) : -1;
        };
        // one step ahead in registers, and the rows' places two ahead
        Regs a, b;
        load(a, c, src, first * NK, mine(first));
        int row = mine(first + stride);
        for (int st = first;;) {
            st += stride;
            if (st < n_steps) load(b, c, src, st * NK, row);
            row = mine(st + stride);
            step(a, scale_log2);
            if (st >= n_steps) break;
            st += stride;
            if (st < n_steps) load(a, c, src, st * NK, row);
            row = mine(st + stride);
            step(b, scale_log2);
            if (st >= n_steps) break;
        }
    }

    // Sums over the quad and adds the zero points: o = sum p v^, l = sum p.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
            l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
            zacc[hr] += __shfl_xor_sync(0xffffffffu, zacc[hr], 1);
            zacc[hr] += __shfl_xor_sync(0xffffffffu, zacc[hr], 2);
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][2 * hr] += zacc[hr];
                o[j][2 * hr + 1] += zacc[hr];
            }
        }
    }

    // Partial (after finish): part[h] = {m, l}, then O rows of D floats at
    // part + 32 (16 heads).
    __device__ __forceinline__ void store_part(float* part, int g) const {
        const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const int h = gid + 8 * hr;
            if (h >= g) continue;
            if (t == 0) {
                part[2 * h] = m[hr];
                part[2 * h + 1] = l[hr];
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

// kv_quant.cu -- writing rows of K and V into a quantised cache, and reading
// them back ("HySparse 混合稀疏注意力（一）" counts its KV caches in FP8; the
// 4-bit rows halve that again).
//
// Row x of head_dim values, in fp32 with IEEE division:
//   HS_KV_INT4: scale = bf16((max - min) / 15), zero = bf16(min),
//               code = clamp(rint((x - zero) / scale), 0, 15);
//   HS_KV_FP8:  scale = bf16(max|x| / 448), zero = 0, code = e4m3(x / scale).
// scale = 0 (a constant row, or a range below bf16's smallest step) has code 0.
// A row with a NaN or an infinity, or whose scale or zero overflows, has both as
// NaN, so that it reads back as NaN.
//
// Both are one pass: D / 8 lanes per row, eight elements each, the row's range
// by shuffles, kRows rows per thread in flight.  Floor: HBM (2 D bytes in, D / 2 + 4 or
// D + 4 out per bf16 row).  The quotients that only pick a code are taken with a
// reciprocal, and by the stated division where that could matter (near a border
// between two codes): 8192 x 4 rows of 128, K and V, 4-bit, 21 MB in and out: 11.7 us written
// (1.8 TB/s; 16.8 us with IEEE division throughout), 5.8 us read back (3.7 TB/s).  The write
// issues 113 warp instructions a row, 6.6 us of the schedulers' time.
#include <cuda_fp8.h>

#include "hs_common.cuh"
#include "hs_kernels.cuh"
#include "quant_kv.cuh"

namespace hs {
namespace kvq {

struct Args {
    KParams p;
    const int32_t* seq_len;  // length after the write; null: q_offset + t_q
    const int32_t* n_new;    // rows of this call; null: t_q
    uint8_t* codes[2];
    uint32_t* entry[2];
    void* x[2];
};
constexpr int kThreads = 128;

// Eight elements as they lie: 4 words of bf16 pairs, or 8 of fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, uint32_t (&w)[sizeof(T) * 2]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint32_t (&w)[sizeof(T) * 2], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * 2; ++i) {
        if constexpr (sizeof(T) == 2) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            x[i] = __uint_as_float(w[i]);
        }
    }
}

__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a),
                                         *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a),
                                         *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Minimum and maximum of the row that LN lanes hold eight elements each of; NaN if it
// holds one.  Both travel as one pair (minimum, - maximum).
template <typename T, int LN>
__device__ __forceinline__ void row_range(const uint32_t (&w)[sizeof(T) * 2], const float (&x)[8],
                                          float& lo, float& hi) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t a = min_nan2(min_nan2(w[0], w[1]), min_nan2(w[2], w[3]));
        const uint32_t b = max_nan2(max_nan2(w[0], w[1]), max_nan2(w[2], w[3])) ^ 0x80008000u;
        uint32_t m = min_nan2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
        for (int s = 1; s < LN; s <<= 1) m = min_nan2(m, __shfl_xor_sync(0xffffffffu, m, s));
        lo = __uint_as_float(m << 16);
        hi = -__uint_as_float(m & 0xffff0000u);
    } else {
        lo = x[0];
        hi = -x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min_nan(lo, x[i]);
            hi = min_nan(hi, -x[i]);
        }
#pragma unroll
        for (int s = 1; s < LN; s <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
            hi = min_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
        }
        hi = -hi;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                  pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// The rows of a block: sequence b, kv head u, rows j0.. of the call.
struct Rows {
    int b, u, bu, j0;
    int n, first;  // rows of the sequence, and row 0's position; n = 0: none

    __device__ __forceinline__ Rows(const Args& a, int per_block) {
        const KParams& p = a.p;
        const int tiles = (p.t_q + per_block - 1) / per_block;
        bu = blockIdx.x / tiles;
        j0 = (blockIdx.x - bu * tiles) * per_block;
        b = bu / p.hkv;
        u = bu - b * p.hkv;
        n = a.n_new ? __ldg(a.n_new + b) : p.t_q;
        const int L = a.seq_len ? __ldg(a.seq_len + b) : p.q_offset + p.t_q;
        first = L - n;
        if (n < 0 || n > p.t_q || L < n || L > p.t_kv) {
            if (threadIdx.x == 0) set_status(HS_ERR_BOUNDS);
            n = 0;
        }
    }
    // Cache row of row j, -1 if there is none.
    __device__ __forceinline__ long long row(const KParams& p, int j) const {
        if (j >= n) return -1;
        if (p.bt) return page_map(p, b, u).row(first + j);
        return (long long)bu * p.t_kv + first + j;
    }
    // Row j of the call's k or v.
    __device__ __forceinline__ long long at(const KParams& p, int j) const {
        return (long long)bu * p.t_q + j;
    }
};

// Codes of a lane's eight elements: 4 bits each in w[0], or 8 in w[0] and w[1].
template <int F>
__device__ __forceinline__ void encode8_exact(const float (&x)[8], float s, float z, uint32_t (&w)[2]) {
    w[0] = w[1] = 0u;
    if (!(s > 0.f)) return;  // constant row, or NaN entry
    if constexpr (F == HS_KV_INT4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], z), s)), 0.f), 15.f);
            w[0] |= (uint32_t)c << (4 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_fp8_storage_t c =
                __nv_cvt_float_to_fp8(__fdiv_rn(x[i], s), __NV_SATFINITE, __NV_E4M3);
            w[i >> 2] |= (uint32_t)c << (8 * (i & 3));
        }
    }
}
// The same codes with y = (x - z) r, r = 1 / s to 2^-22, in place of the quotient: false if a
// quotient may lie on the other side of a border between two codes than y does.
template <int F, bool kClamp>
__device__ __forceinline__ bool encode8_near(const float (&x)[8], float r, float z, uint32_t (&w)[2]) {
    w[0] = w[1] = 0u;
    if constexpr (F == HS_KV_INT4) {
        constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer
        float far = 0.f, d[8];
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            float y = (x[i] - z) * r;
            // bf16 rows: zero is their minimum itself, and 15 scale at least their range
            // less 2^-9 of it, so 0 <= y < 15.1
            if constexpr (kClamp) y = fminf(fmaxf(y, 0.f), 15.f);
            const float c = y + kMagic;
            d[i] = fabsf(y - (c - kMagic));
            w[0] = w[0] * 16u + __float_as_uint(c);
        }
        // what the magic number's bits added up to
        constexpr uint32_t kBits = 0x4b400000u;
        w[0] -= kBits * 0x11111111u;
#pragma unroll
        for (int i = 0; i < 8; i += 2) far = tc::max3f(far, d[i], d[i + 1]);
        return far < 0.49998f;  // y is off by less than 1e-5
    } else {
        uint32_t v[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float a = x[i] * r, b = x[i + 1] * r;
            constexpr float kDown = 1.f - 0x1p-21f, kUp = 1.f + 0x1p-21f;
            w[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a * kDown, b * kDown),
                                                            __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
            v[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a * kUp, b * kUp),
                                                            __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
        }
        return w[0] == v[0] && w[1] == v[1];
    }
}

template <int D, int F, typename T, int kRows>
__global__ void __launch_bounds__(kThreads) kv_quant_write_kernel(Args a) {
    constexpr int LN = D / 8, PASS = kThreads / LN;  // lanes per row, rows per pass
    const Rows rows(a, PASS * kRows);
    const int c = threadIdx.x % LN, side = blockIdx.y;
    const T* src = (const T*)a.x[side];
    uint32_t raw[kRows][sizeof(T) * 2];
    const int j0 = rows.j0 + threadIdx.x / LN;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int j = j0 + k * PASS;
        if (j < rows.n) {
            load8(src + rows.at(a.p, j) * D + c * 8, raw[k]);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) * 2; ++i) raw[k][i] = 0u;
        }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        float x[8];
        unpack8<T>(raw[k], x);
        float lo, hi;
        row_range<T, LN>(raw[k], x, lo, hi);
        float s, z;
        if constexpr (F == HS_KV_INT4) {
            s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
            z = __bfloat162float(__float2bfloat16_rn(lo));
        } else {
            s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(fmaxf(fabsf(lo), fabsf(hi)), 448.f)));
            z = 0.f;
        }
        if (!isfinite(s) || !isfinite(z) || lo != lo) s = z = __int_as_float(0x7fc00000);
        const long long row = rows.row(a.p, j0 + k * PASS);
        if (row < 0) continue;
        uint32_t w[2];
        // a reciprocal that is a normal number, and quotients that fit
        if (!(s > 1e-30f && s < 1e30f) || !encode8_near<F, sizeof(T) != 2>(x, __frcp_rn(s), z, w))
            encode8_exact<F>(x, s, z, w);
        if constexpr (F == HS_KV_INT4)
            *reinterpret_cast<uint32_t*>(a.codes[side] + row * (D / 2) + c * 4) = w[0];
        else
            *reinterpret_cast<uint2*>(a.codes[side] + row * D + c * 8) = make_uint2(w[0], w[1]);
        if (c == 0) a.entry[side][row] = pack_bf16(s, z);
    }
}

template <int D, int F, typename T, int kRows>
__global__ void __launch_bounds__(kThreads) kv_quant_read_kernel(Args a) {
    constexpr int LN = D / 8, PASS = kThreads / LN;
    const Rows rows(a, PASS * kRows);
    const int c = threadIdx.x % LN, side = blockIdx.y;
    const int j0 = rows.j0 + threadIdx.x / LN;
    uint2 w[kRows];
    uint32_t e[kRows];
    bool live[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const long long row = rows.row(a.p, j0 + k * PASS);
        live[k] = row >= 0;
        if (!live[k]) continue;
        e[k] = __ldg(a.entry[side] + row);
        if constexpr (F == HS_KV_INT4)
            w[k].x = __ldg(reinterpret_cast<const uint32_t*>(a.codes[side] + row * (D / 2)) + c);
        else
            w[k] = __ldg(reinterpret_cast<const uint2*>(a.codes[side] + row * D) + c);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        if (!live[k]) continue;
        const float s = entry_scale(e[k]), z = entry_zero(e[k]);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (F == HS_KV_INT4) {
                x[i] = fmaf((float)((w[k].x >> (4 * i)) & 15u), s, z);
            } else {
                const uint32_t b = ((i < 4 ? w[k].x : w[k].y) >> (8 * (i & 3))) & 255u;
                const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
                x[i] = fmaf(__half2float(__half(h)), s, z);
            }
        }
        store8((T*)a.x[side] + rows.at(a.p, j0 + k * PASS) * D + c * 8, x);
    }
}

template <int D, int F, typename T, int kRows>
static void launch_r(const Args& a, bool write, cudaStream_t st) {
    constexpr int per_block = kThreads / (D / 8) * kRows;
    const dim3 grid((unsigned)a.p.batch * a.p.hkv * ((a.p.t_q + per_block - 1) / per_block), 2);
    if (write) kv_quant_write_kernel<D, F, T, kRows><<<grid, kThreads, 0, st>>>(a);
    else kv_quant_read_kernel<D, F, T, kRows><<<grid, kThreads, 0, st>>>(a);
}

template <int D, int F, typename T>
static void launch_t(const Args& a, bool write, cudaStream_t st) {
    // Several rows per thread once a (sequence, kv head)'s rows fill such a block (8192 x 4
    // rows: write 16.8 -> 13.5 us, read 8.5 -> 5.8 us, with four); one token's take one.
    if (a.p.t_q >= 4 * (kThreads / (D / 8))) launch_r<D, F, T, 4>(a, write, st);
    else launch_r<D, F, T, 1>(a, write, st);
}

template <int D, int F>
static void launch_d(const Args& a, int dtype, bool write, cudaStream_t st) {
    if (dtype == HS_BF16) launch_t<D, F, __nv_bfloat16>(a, write, st);
    else launch_t<D, F, float>(a, write, st);
}

}  // namespace kvq

cudaError_t launch_kv_quant(const KParams& p, int dtype, int format, void* k_codes, void* k_entry,
                            void* v_codes, void* v_entry, void* k, void* v,
                            const int32_t* seq_len, const int32_t* n_new, bool write,
                            cudaStream_t st) {
    kvq::Args a;
    a.p = p;
    a.seq_len = seq_len;
    a.n_new = n_new;
    a.codes[0] = (uint8_t*)k_codes;
    a.codes[1] = (uint8_t*)v_codes;
    a.entry[0] = (uint32_t*)k_entry;
    a.entry[1] = (uint32_t*)v_entry;
    a.x[0] = k;
    a.x[1] = v;
    if (format == HS_KV_INT4) {
        if (p.head_dim == 64) kvq::launch_d<64, HS_KV_INT4>(a, dtype, write, st);
        else kvq::launch_d<128, HS_KV_INT4>(a, dtype, write, st);
    } else {
        if (p.head_dim == 64) kvq::launch_d<64, HS_KV_FP8>(a, dtype, write, st);
        else kvq::launch_d<128, HS_KV_FP8>(a, dtype, write, st);
    }
    return cudaGetLastError();
}

}  // namespace hs

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
// by shuffles, kRows rows per thread in flight.  Bound: HBM (2 D bytes in, D / 2 + 4 or
// D + 4 out per bf16 row).  The quotients that only pick a code are taken with a
// reciprocal, and by the stated division where that could matter (near a border
// between two codes): XXX
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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
            x[4 * i] = v.x;
            x[4 * i + 1] = v.y;
            x[4 * i + 2] = v.z;
            x[4 * i + 3] = v.w;
        }
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
template <int F>
__device__ __forceinline__ bool encode8_near(const float (&x)[8], float r, float z, uint32_t (&w)[2]) {
    w[0] = w[1] = 0u;
    if constexpr (F == HS_KV_INT4) {
        constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = fminf(fmaxf((x[i] - z) * r, 0.f), 15.f);
            const float c = y + kMagic;
            far = fmaxf(far, fabsf(y - (c - kMagic)));
            w[0] |= (__float_as_uint(c) & 15u) << (4 * i);
        }
        return far < 0.49998f;  // y <= 15 is off by less than 1e-5
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
    float x[kRows][8];
    const int j0 = rows.j0 + threadIdx.x / LN;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int j = j0 + k * PASS;
        if (j < rows.n) {
            load8(src + rows.at(a.p, j) * D + c * 8, x[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = 0.f;
        }
    }
    const uint32_t seg = ((1u << (LN & 31)) - 1u) << ((threadIdx.x & 31) / LN * LN);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        float lo = x[k][0], hi = x[k][0], sum = 0.f;  // sum: a NaN or an infinity shows in it
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, x[k][i]);
            hi = fmaxf(hi, x[k][i]);
            sum = fmaf(x[k][i], 0.f, sum);
        }
#pragma unroll
        for (int m = 1; m < LN; m <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
        }
        const bool bad = (__ballot_sync(0xffffffffu, sum != 0.f) & seg) != 0u;
        float s, z;
        if constexpr (F == HS_KV_INT4) {
            s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)));
            z = __bfloat162float(__float2bfloat16_rn(lo));
        } else {
            s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(fmaxf(fabsf(lo), fabsf(hi)), 448.f)));
            z = 0.f;
        }
        if (bad || !isfinite(s) || !isfinite(z)) s = z = __int_as_float(0x7fc00000);
        const long long row = rows.row(a.p, j0 + k * PASS);
        if (row < 0) continue;
        uint32_t w[2];
        // a reciprocal that is a normal number, and quotients that fit
        if (!(s > 1e-30f && s < 1e30f) || !encode8_near<F>(x[k], __frcp_rn(s), z, w))
            encode8_exact<F>(x[k], s, z, w);
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
    // several rows per thread once they fill the blocks of a few rows per SM
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

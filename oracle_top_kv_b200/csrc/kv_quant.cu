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
// by shuffles.  Bound: HBM (2 D bytes in, D / 2 + 4 or D + 4 out per bf16 row).
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
    long long rows;          // batch * hkv * t_q
};

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

// Cache row of row r = (b, u, j) of the call, -1 if there is none.
__device__ __forceinline__ long long cache_row(const Args& a, long long r) {
    const KParams& p = a.p;
    const int j = (int)(r % p.t_q);
    const long long bu = r / p.t_q;
    const int u = (int)(bu % p.hkv), b = (int)(bu / p.hkv);
    const int n = a.n_new ? __ldg(a.n_new + b) : p.t_q;
    const int L = a.seq_len ? __ldg(a.seq_len + b) : p.q_offset + p.t_q;
    if (n < 0 || n > p.t_q || L < n || L > p.t_kv) {
        set_status(HS_ERR_BOUNDS);
        return -1;
    }
    if (j >= n) return -1;
    const int pos = L - n + j;
    if (p.bt) return page_map(p, b, u).row(pos);
    return bu * p.t_kv + pos;
}

// Codes of a lane's eight elements: 4 bits each in w[0], or 8 in w[0] and w[1].
template <int F>
__device__ __forceinline__ void encode8(const float (&x)[8], float s, float z, uint32_t (&w)[2]) {
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

template <int D, int F, typename T>
__global__ void __launch_bounds__(256) kv_quant_write_kernel(Args a) {
    constexpr int LN = D / 8;  // lanes per row
    const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / LN;
    const int c = threadIdx.x % LN, side = blockIdx.y;
    const long long row = r < a.rows ? cache_row(a, r) : -1;
    float x[8];
    if (row >= 0) {
        load8((const T*)a.x[side] + r * D + c * 8, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    float lo = x[0], hi = x[0];
    bool bad = !isfinite(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad |= !isfinite(x[i]);
    }
#pragma unroll
    for (int m = 1; m < LN; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const uint32_t seg = (LN == 32 ? 0xffffffffu : ((1u << (LN & 31)) - 1u))
                         << ((threadIdx.x & 31) / LN * LN);
    bad = (__ballot_sync(0xffffffffu, bad) & seg) != 0u;
    if (row < 0) return;
    float s, z;
    if constexpr (F == HS_KV_INT4) {
        const float range = __fsub_rn(hi, lo);
        s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(range, 15.f)));
        z = __bfloat162float(__float2bfloat16_rn(lo));
    } else {
        s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(fmaxf(fabsf(lo), fabsf(hi)), 448.f)));
        z = 0.f;
    }
    if (bad || !isfinite(s) || !isfinite(z)) s = z = __int_as_float(0x7fc00000);
    uint32_t w[2];
    encode8<F>(x, s, z, w);
    if constexpr (F == HS_KV_INT4)
        *reinterpret_cast<uint32_t*>(a.codes[side] + row * (D / 2) + c * 4) = w[0];
    else
        *reinterpret_cast<uint2*>(a.codes[side] + row * D + c * 8) = make_uint2(w[0], w[1]);
    if (c == 0) a.entry[side][row] = pack_bf16(s, z);
}

template <int D, int F, typename T>
__global__ void __launch_bounds__(256) kv_quant_read_kernel(Args a) {
    constexpr int LN = D / 8;
    const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / LN;
    const int c = threadIdx.x % LN, side = blockIdx.y;
    const long long row = r < a.rows ? cache_row(a, r) : -1;
    if (row < 0) return;
    const uint32_t e = __ldg(a.entry[side] + row);
    const float s = entry_scale(e), z = entry_zero(e);
    float x[8];
    if constexpr (F == HS_KV_INT4) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(a.codes[side] + row * (D / 2)) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((w >> (4 * i)) & 15u), s, z);
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.codes[side] + row * D) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 255u;
            const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
            x[i] = fmaf(__half2float(__half(h)), s, z);
        }
    }
    store8((T*)a.x[side] + r * D + c * 8, x);
}

template <int D, int F, typename T>
static void launch_t(const Args& a, bool write, cudaStream_t st) {
    const long long threads = a.rows * (D / 8);
    const dim3 grid((unsigned)((threads + 255) / 256), 2);
    if (write) kv_quant_write_kernel<D, F, T><<<grid, 256, 0, st>>>(a);
    else kv_quant_read_kernel<D, F, T><<<grid, 256, 0, st>>>(a);
}

template <int D, int F>
static void launch_d(const Args& a, int dtype, bool write, cudaStream_t st) {
    if (dtype == HS_BF16) launch_t<D, F, __nv_bfloat16>(a, write, st);
    else launch_t<D, F, float>(a, write, st);
}

}  // namespace kvq

// Rows whose thread count would not fit the grid.
bool kv_quant_supported(const KParams& p) {
    return (double)p.batch * p.hkv * p.t_q * (p.head_dim / 8) < 256.0 * 2147483647.0;
}

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
    a.rows = (long long)p.batch * p.hkv * p.t_q;
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

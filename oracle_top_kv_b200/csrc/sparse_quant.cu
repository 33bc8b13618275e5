// sparse_quant.cu -- the sparse layers over a quantised K^F/V^F: attention of
// a layer's own query over the rows of an index set, read as codes
// (quant_kv.cuh).  Prefill: one warp per (query row, KV group).  Decode: one
// thread-block cluster per (sequence, KV group); the unit's rows are dealt to
// its warps in steps, partials are merged per CTA in shared memory and over
// the cluster in distributed shared memory.
#include <type_traits>

#include "hs_common.cuh"
#include "hs_kernels.cuh"
#include "quant_kv.cuh"

namespace hs {
namespace sq {

constexpr int kWarps = 4;      // of a decode CTA
constexpr int kRowWarps = 1;   // of a prefill CTA: the warps work alone
constexpr int kStages = 2;
// 16 heads: Q in shared memory leaves registers for 12 warps on an SM in place of 8 (4-bit,
// 2048 rows x 4 groups x 1024 keys: 388 us against 483 with Q in registers, when this was
// chosen; 330 us now).  32 keys a step, of 128-byte rows too, where the work of a step that is
// not its keys' would weigh twice (8-bit, 1000 rows x 8 groups of 4 heads x 16 blocks of 64:
// 297 us with 16 keys a step, 222 to 228 with 32: 9.5 TB/s of rows, most of them from L2).
template <int D, int F, int NH> using Attend = QAttend<D, F, NH, kStages, NH == 2, 32>;
template <int D, int F, int NH>
constexpr size_t kWarpBytes =  // a warp's ring and query
    Attend<D, F, NH>::Ring::kBytes + QQuery<D, F, NH, NH == 2>::kBytes;
// Warps to an SM that the registers are divided for.  8 heads: 14, between few warps and
// few registers (1000 rows x 8 groups of 4 heads, 1024 keys, at 12, 14, 16 warps: 8-bit
// blocks 221, 222, 239 us, 4-bit tokens 231, 213, 219, head_dim 64 163, 148, 149).  Of 8-bit
// rows of 128 the rings take 17 KB a warp (21 with 16 heads' queries): shared memory holds
// 12 warps (10), and the 8-bit figures compare register limits only.
template <int NH> constexpr int kPerSm = NH == 1 ? 14 : 12;

// Writes a unit's heads from a warp's finished accumulators.
template <int D, int NH, class A>
__device__ __forceinline__ void store_rows(const A& st, int g, __nv_bfloat16* o, float* lse,
                                           size_t head0, size_t stride) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = 8 * n + 2 * t + e;
            if (h >= g) continue;
            const float l = e ? st.l[n].y : st.l[n].x;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t row = head0 + h * stride;
            __nv_bfloat16* dst = o + row * D + gid * (D / 8);
#pragma unroll
            for (int x = 0; x < D / 8; x += 8) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = pack_bf16(st.dim(n, e, x + 2 * i) * inv, st.dim(n, e, x + 2 * i + 1) * inv);
                *reinterpret_cast<uint4*>(dst + x) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (gid == 0) {
                const float m = e ? st.m[n].y : st.m[n].x;
                lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            }
        }
}

template <int D, int F, int NH>
__global__ void __launch_bounds__(kRowWarps * 32, kPerSm<NH> / kRowWarps)
    sparse_quant_kernel(KParams p, QuantCache cache, const __nv_bfloat16* __restrict__ q,
                        const int32_t* __restrict__ idx, const int32_t* __restrict__ cnt,
                        __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
    const long long task = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (task >= (long long)p.batch * p.hkv * p.t_q) return;
    const int j = (int)(task % p.t_q);
    const int unit = (int)(task / p.t_q);
    const int u = unit % p.hkv, b = unit / p.hkv;
    const size_t head0 = ((size_t)b * p.hq + (size_t)u * p.group) * p.t_q + j;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    using A = Attend<D, F, NH>;
    const typename A::Ring ring{smem_u32(smem_raw) + (threadIdx.x >> 5) * A::Ring::kBytes};
    A st;
    st.init(q + head0 * D, (size_t)p.t_q * D, p.group, p.scale_log2,
            smem_u32(smem_raw) + kRowWarps * A::Ring::kBytes + (threadIdx.x >> 5) * decltype(st.q)::kBytes);
    const int n = clamp_count(cnt[task], p.ksel) * p.block_size;
    const QIndex<A::NK> src{idx + (size_t)task * p.ksel, n, p.block_size, p.q_offset + j,
                            page_map(p, b, u)};
    st.run(ring, unit_cache<D, F>(p, cache, unit), src, 0, 1, (n + A::NK - 1) / A::NK, NoMaxima{});
    st.finish();
    store_rows<D, NH>(st, p.group, o, lse, head0, (size_t)p.t_q);
}

// Weight of a partial with reference m under the common reference M.
__device__ __forceinline__ float merge_weight(float m, float M) {
    return m == -INFINITY ? 0.f : exp2f(m - M);
}

// Four fp32 at shared address `a` of cluster CTA `rank`.
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t a, uint32_t rank) {
    uint32_t ra;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(ra)
                 : "memory");
    return v;
}

template <int D, int F, int NH>
__global__ void __launch_bounds__(kWarps * 32, kPerSm<NH> / kWarps)
    decode_sparse_quant_kernel(KParams p, QuantCache cache, const __nv_bfloat16* __restrict__ q,
                               const int32_t* __restrict__ seq_len,
                               const int32_t* __restrict__ idx, const int32_t* __restrict__ cnt,
                               int csize, __nv_bfloat16* __restrict__ o,
                               float* __restrict__ lse) {
    using A = Attend<D, F, NH>;
    // the warps' rings, reused for their partials; then the CTA's partial
    extern __shared__ __align__(16) unsigned char smem_raw[];
    constexpr int kStride = A::Ring::kBytes / 4;  // floats between the warps' partials
    static_assert(kStride >= A::kPart, "a partial fits a ring");
    float* smem = reinterpret_cast<float*>(smem_raw);
    const int warp = threadIdx.x >> 5, g = p.group;
    const int crank = csize > 1 ? (int)cluster_rank() : 0;
    const int unit = blockIdx.x / csize;
    const int u = unit % p.hkv, b = unit / p.hkv;
    const int L = seq_len[b];
    const bool valid = L >= 1 && L <= p.t_kv;
    const size_t head0 = (size_t)b * p.hq + (size_t)u * g;
    A st;
    st.init(q + head0 * D, D, g, p.scale_log2,
            smem_u32(smem_raw) + kWarps * A::Ring::kBytes + warp * decltype(st.q)::kBytes);
    const typename A::Ring ring{smem_u32(smem_raw) + warp * A::Ring::kBytes};
    if (valid) {
        const int n = clamp_count(cnt[unit], p.ksel);
        const QIndex<A::NK> src{idx + (size_t)unit * p.ksel, n, 1, L - 1, page_map(p, b, u)};
        st.run(ring, unit_cache<D, F>(p, cache, unit), src, crank * kWarps + warp, kWarps * csize,
               (n + A::NK - 1) / A::NK, NoMaxima{});
    } else if (crank == 0 && threadIdx.x == 0) {
        set_status(HS_ERR_BOUNDS);
    }
    st.finish();
    st.store_part(smem + warp * kStride, g);
    __syncthreads();
    // the CTA's partial: weights of the warps' first, then the sums
    float* mine = smem + kWarps * kWarpBytes<D, F, NH> / sizeof(float);
    __shared__ float s_f[8][16], s_scale[16];  // weights per (warp, then CTA) and head
    const int h16 = threadIdx.x & 15, w16 = threadIdx.x >> 4;
    if (w16 < kWarps && h16 < g) {
        float m[kWarps], M = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m[w] = smem[w * kStride + 2 * h16]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += smem[w * kStride + 2 * h16 + 1] * merge_weight(m[w], M);
        s_f[w16][h16] = merge_weight(smem[w16 * kStride + 2 * h16], M);
        if (w16 == 0) {
            mine[2 * h16] = M;
            mine[2 * h16 + 1] = l;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < g * (D / 4); e += blockDim.x) {
        const int h = e / (D / 4);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_f[w][h];
            const float4 x = reinterpret_cast<const float4*>(smem + w * kStride + 32)[e];
            a.x += x.x * f;
            a.y += x.y * f;
            a.z += x.z * f;
            a.w += x.w * f;
        }
        reinterpret_cast<float4*>(mine + 32)[e] = a;
    }
    __syncwarp();  // the barrier takes whole warps
    if (csize > 1) cluster_sync_all();
    else __syncthreads();
    // the cluster's: weights again, then each CTA writes a share of the outputs
    const uint32_t at = smem_u32(mine);
    if (w16 < csize && h16 < g) {
        float M = -INFINITY, l = 0.f;
        for (int r = 0; r < csize; ++r) M = fmaxf(M, ld_cluster_f32(at + 8u * h16, (uint32_t)r));
        for (int r = 0; r < csize; ++r)
            l += ld_cluster_f32(at + 8u * h16 + 4u, (uint32_t)r) *
                 merge_weight(ld_cluster_f32(at + 8u * h16, (uint32_t)r), M);
        s_f[w16][h16] = merge_weight(ld_cluster_f32(at + 8u * h16, (uint32_t)w16), M);
        if (w16 == 0) {
            s_scale[h16] = l == 0.f ? 0.f : 1.f / l;
            if (crank == 0 && lse) lse[head0 + h16] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
        }
    }
    __syncthreads();
    for (int e = crank * blockDim.x + threadIdx.x; e < g * (D / 4); e += csize * blockDim.x) {
        const int h = e / (D / 4);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < csize; ++r) {
            const float f = s_f[r][h];
            const float4 x = ld_cluster_f32x4(at + 128u + 16u * e, (uint32_t)r);
            a.x += x.x * f;
            a.y += x.y * f;
            a.z += x.z * f;
            a.w += x.w * f;
        }
        const float inv = s_scale[h];
        *reinterpret_cast<uint2*>(o + head0 * D + 4 * e) =
            make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    }
    __syncwarp();
    if (csize > 1) cluster_sync_all();  // peers keep their shared memory until all have read
}

template <int D, int F, int NH>
static cudaError_t launch_sparse_t(const KParams& p, const QuantCache& c, const void* q,
                                   const int32_t* idx, const int32_t* cnt, void* o, float* lse,
                                   cudaStream_t st) {
    const long long tasks = (long long)p.batch * p.hkv * p.t_q;
    auto kern = sparse_quant_kernel<D, F, NH>;
    constexpr int smem = kRowWarps * (int)kWarpBytes<D, F, NH>;
    static_assert(smem <= 48 * 1024, "more needs the kernel's attribute set");
    kern<<<(unsigned)((tasks + kRowWarps - 1) / kRowWarps), kRowWarps * 32, smem, st>>>(
        p, c, (const __nv_bfloat16*)q, idx, cnt, (__nv_bfloat16*)o, lse);
    return cudaGetLastError();
}

template <int D, int F, int NH>
static cudaError_t launch_decode_t(const KParams& p, const QuantCache& c, const void* q,
                                   const int32_t* seq_len, const int32_t* idx, const int32_t* cnt,
                                   void* o, float* lse, cudaStream_t st) {
    auto kern = decode_sparse_quant_kernel<D, F, NH>;
    const size_t smem = kWarps * kWarpBytes<D, F, NH> + Attend<D, F, NH>::kPart * sizeof(float);
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    // Widest cluster (a portable size) whose CTAs still run in one wave, two
    // to an SM, with a step for every warp (8 units of 1152 rows: 8.8 us on clusters of 8,
    // 19 on one CTA each; 128 units of 1024 rows: 18.4 us on pairs, as on one).
    const int units = p.batch * p.hkv;
    const int steps = (p.ksel + Attend<D, F, NH>::NK - 1) / Attend<D, F, NH>::NK;
    int csize = 1;
    while (csize < 8 && units * csize * 2 <= 2 * sms && kWarps * csize < steps) csize *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(units * csize));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p, c, (const __nv_bfloat16*)q, seq_len, idx, cnt, csize,
                              (__nv_bfloat16*)o, lse);
}

// Calls fn.operator()<D, F, NH>(): NH 8-head tiles hold the group.
template <typename Fn>
static cudaError_t dispatch(const KParams& p, int format, Fn fn) {
    auto by_g = [&](auto d, auto f) {
        constexpr int D = decltype(d)::value, F = decltype(f)::value;
        return p.group <= 8 ? fn.template operator()<D, F, 1>() : fn.template operator()<D, F, 2>();
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    using F4 = std::integral_constant<int, HS_KV_INT4>;
    using F8 = std::integral_constant<int, HS_KV_FP8>;
    if (format == HS_KV_INT4) return p.head_dim == 64 ? by_g(I64{}, F4{}) : by_g(I128{}, F4{});
    return p.head_dim == 64 ? by_g(I64{}, F8{}) : by_g(I128{}, F8{});
}

struct SparseLaunch {
    const KParams& p;
    const QuantCache& c;
    const void* q;
    const int32_t *seq_len, *idx, *cnt;  // seq_len: a decode step
    void* o;
    float* lse;
    cudaStream_t st;
    template <int D, int F, int NH>
    cudaError_t operator()() const {
        return seq_len ? launch_decode_t<D, F, NH>(p, c, q, seq_len, idx, cnt, o, lse, st)
                       : launch_sparse_t<D, F, NH>(p, c, q, idx, cnt, o, lse, st);
    }
};

}  // namespace sq

cudaError_t launch_sparse_quant(const KParams& p, int format, const QuantCache& c, const void* q,
                                const int32_t* idx, const int32_t* cnt, void* o, float* lse,
                                cudaStream_t st) {
    return sq::dispatch(p, format, sq::SparseLaunch{p, c, q, nullptr, idx, cnt, o, lse, st});
}

cudaError_t launch_decode_sparse_quant(const KParams& p, int format, const QuantCache& c,
                                       const void* q, const int32_t* seq_len, const int32_t* idx,
                                       const int32_t* cnt, void* o, float* lse, cudaStream_t st) {
    return sq::dispatch(p, format, sq::SparseLaunch{p, c, q, seq_len, idx, cnt, o, lse, st});
}

}  // namespace hs

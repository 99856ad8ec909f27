// fp8_quant.hip — activations to OCP e4m3 codes with one fp32 scale per row and
// 128 columns (Fp8Rule, fp8.h).
//
// HBM-bound: T*H*(size + 1) + T*H/32 bytes.  Sixteen lanes hold one block,
// eight values each (16-byte loads of 16-bit inputs, two of fp32), so the
// block's maximum is four DPP steps inside a row of lanes and a lane's codes
// are one 8-byte store.  A wave takes kFp8QuantIters groups of four blocks,
// all loads issued before the first reduction.  4,096 x 2048 bf16: 6.4 us,
// 3.95 TB/s (5.3 us at the rate of a large copy).
#include "fp8.h"

namespace moe {

namespace {

constexpr int kFp8QuantIters = 2;


__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <typename XT>   // _Float16 or __bf16
__device__ __forceinline__ void load8(const XT* p, float (&v)[8]) {
    typedef XT x8 __attribute__((ext_vector_type(8)));
    const x8 a = *reinterpret_cast<const x8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
}

// Maximum of unsigned values over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
    v = max(v, dpp_u<0xB1>(v));
    v = max(v, dpp_u<0x4E>(v));
    v = max(v, dpp_u<0x141>(v));
    return max(v, dpp_u<0x140>(v));
}

// Lane group (16 lanes) number `grp` of the launch takes blocks grp, grp + stride, ...
template <typename XT>
__device__ __forceinline__ void quantize_fp8_lanes(int64_t grp, int64_t stride, const XT* __restrict__ x, int64_t ldx,
                                                   int64_t n_blocks, int nb, int H, uint8_t* __restrict__ xq,
                                                   float* __restrict__ xs) {
    const int l = threadIdx.x & 15;
    float v[kFp8QuantIters][8];
    int64_t row[kFp8QuantIters];
    int col[kFp8QuantIters];
#pragma unroll
    for (int i = 0; i < kFp8QuantIters; ++i) {
        const int64_t b = grp + i * stride;
        row[i] = b / nb;
        col[i] = (int)(b - row[i] * nb) * kFp8Block + 8 * l;
        if (b < n_blocks && col[i] < H)
            load8(x + row[i] * ldx + col[i], v[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kFp8QuantIters; ++i) {
        const int64_t b = grp + i * stride;
        uint32_t m = 0;   // |x| orders as its bit pattern, infinities and NaN above every finite value
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        m = row16_max_u32(m);
        const bool fin = m < 0x7F800000u;
        if (b >= n_blocks) continue;
        const Fp8Rule rule(__uint_as_float(fin ? m : 0u));
        uint2 q;
        q.x = rule.pack4(v[i][0], v[i][1], v[i][2], v[i][3]);
        q.y = rule.pack4(v[i][4], v[i][5], v[i][6], v[i][7]);
        if (!fin) {
            q = make_uint2(0u, 0u);
            if (l == 0) raise_error(kErrActNonFinite);
        }
        if (col[i] < H) *reinterpret_cast<uint2*>(xq + row[i] * H + col[i]) = q;
        if (l == 0) xs[b] = rule.d;
    }
}

// The quantiser's work, in workgroups of 1,024 threads (alone, or carried by the routing launches of a layer call).
template <typename XT>
struct ActQuant {
    static constexpr int kGroups = 1024 / 16;
    const XT* x = nullptr;
    int64_t ldx = 0, n_blocks = 0;
    int nb = 1, H = 0;
    uint8_t* xq = nullptr;
    float* xs = nullptr;
    ActQuant() = default;
    ActQuant(const void* x_, int64_t ldx_, int T, int H_, uint8_t* xq_, float* xs_)
        : x((const XT*)x_), ldx(ldx_), nb((H_ + kFp8Block - 1) / kFp8Block), H(H_), xq(xq_), xs(xs_) {
        n_blocks = (int64_t)T * nb;
    }
    unsigned groups() const {
        return (unsigned)((n_blocks + kGroups * kFp8QuantIters - 1) / (kGroups * kFp8QuantIters));
    }
    __device__ __forceinline__ void run(int wg) const {
        quantize_fp8_lanes<XT>((int64_t)wg * kGroups * kFp8QuantIters + threadIdx.x / 16, kGroups, x, ldx, n_blocks, nb, H,
                               xq, xs);
    }
};

template <typename XT>
__global__ void __launch_bounds__(1024) quantize_fp8_kernel(const ActQuant<XT> q) {
    q.run(blockIdx.x);
}

template <typename XT>
hipError_t launch_quantize_fp8_t(const ActQuant<XT>& q, hipStream_t s) {
    quantize_fp8_kernel<XT><<<q.groups(), 1024, 0, s>>>(q);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const void* x, ElemType xt, int64_t ldx, int T, int H, uint8_t* xq, float* xs,
                               hipStream_t s) {
    if (xt == ElemType::kF32) return launch_quantize_fp8_t(ActQuant<float>(x, ldx, T, H, xq, xs), s);
    if (xt == ElemType::kF16) return launch_quantize_fp8_t(ActQuant<_Float16>(x, ldx, T, H, xq, xs), s);
    return launch_quantize_fp8_t(ActQuant<__bf16>(x, ldx, T, H, xq, xs), s);
}

}  // namespace moe

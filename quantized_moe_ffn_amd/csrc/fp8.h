// fp8.h — internal launchers and device helpers of the scored routing and the
// 8-bit float (OCP e4m3) path: quantiser, block-scaled products, expert layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"
#include "kernels.h"

namespace moe {

// ------------------------------------------------------------------ scored routing

struct ScoreRule {
    int sigmoid;        // 0: softmax over the E logits, 1: sigmoid of each
    int n_group;        // 1: no groups
    int topk_group;
    int group_top;      // a group's score: the sum of its 1 or 2 largest biased scores
    int renorm;
    float scale;
    const float* bias;  // [E] or null
};

hipError_t launch_route_scored(const float* logits, int T, int E, int k, const ScoreRule& rule, const RoutingPtrs& r,
                               void* ws, hipStream_t s);

// ------------------------------------------------------------------ 8-bit float path

constexpr int kFp8Block = 128;

enum class ElemType { kF32, kF16, kBF16 };

// One e4m3 matrix bank: n matrices of rows x cols codes, one fp32 scale per
// 128 x 128 block.
struct Fp8Mat {
    const uint8_t* data;
    const float* scale;
    int64_t row_stride, expert_stride;   // bytes
    int rows, cols;
};

hipError_t launch_quantize_fp8(const void* x, ElemType xt, int64_t ldx, int T, int H, uint8_t* xq, float* xs,
                               hipStream_t s);

// The grouped products' work list: tile i of expert e covers rows mt*i .. of its
// bucket; the shared expert's tiles (e = E) cover all T tokens.  row0 is the
// tile's first row of h: its position in the bucket order, or T*k + m0.
struct Fp8Item {
    int e, m0, n_tok, row0;
};
struct Fp8ItemList {
    Fp8Item* items;
    int32_t* n_items;
    int mt;                  // tokens per tile; 0: no list
    int max_items;
    int T;
    int has_shared;
};

// A layer call's routing: launch_route_scored, x [T][H] quantised by extra workgroups of the same launch and, with
// tl.mt > 0, the grouped products' work list; *list_done says whether that was written.
hipError_t launch_route_quantize_fp8(const float* logits, int T, int E, int k, const ScoreRule& rule,
                                     const RoutingPtrs& r, void* ws, const Fp8ItemList& tl, const void* x, ElemType xt, int H,
                                     uint8_t* xq, float* xs, hipStream_t s, bool* list_done);

struct Fp8MatmulArgs {
    const uint8_t* xq;
    const float* xs;
    Fp8Mat w;
    void* y;
    ElemType yt;
    int64_t ldy;
    int T;
};
hipError_t launch_matmul_fp8(const Fp8MatmulArgs& a, hipStream_t s);

struct Fp8FfnArgs {
    Fp8Mat gate, up, down, sgate, sup, sdown;
    int has_shared, H, I, T, k, E;
    RoutingPtrs r;
    const uint8_t* xq;       // [T][H]
    const float* xs;         // [T][H/128]
    uint8_t* hq;             // workspace [T*k (+T)][I], bucket order, then the shared expert's rows
    float* hs;               // workspace [T*k (+T)][I/128]
    void* y_pair;            // [T*k][H] fp32, or fp16 with scales (pair16)
    void* y_shared;          // [T][H], the same
    float* y_scale;          // pair16: [T*k (+T)][H/64]
    int pair16;
    int exact;               // products with fp32 sums throughout (fp8_gemm.hip)
    void* tiles;             // workspace: the work list (fp8_items_bytes), 16-byte aligned
    float* hf;               // workspace of the few-pair kernels: h in fp32, [T*k (+T)][I]
};
size_t fp8_items_bytes(int T, int k, int E, int has_shared);
Fp8ItemList fp8_item_list(const Fp8FfnArgs& f);   // the list launch_ffn_fp8 works through, in f.tiles
hipError_t launch_ffn_fp8(const Fp8FfnArgs& a, bool list_done, hipStream_t s);

// Few pairs: T*k up to this, and up to the expert count, so that few pairs share an expert's read.
constexpr int kFewPairs = 64;
constexpr int kMaxSlots = 17;   // top-k and the shared expert
inline bool fp8_few_pairs(int T, int k, int E) { return T * k <= kFewPairs && T * k <= E; }

struct Fp8CombineArgs {
    const void* y_pair;      // [T*k][H] fp32, or fp16 with scales (pair16)
    const void* y_shared;    // [T][H], the same, or null
    const float* y_scale;    // pair16: [T*k (+T)][H/64]
    int pair16;
    const float* w;          // [T][k]
    const float* shared_scale;
    void* out;
    ElemType ot;
    int T, k, H;
};
// c.out null: y_pair and y_shared (fp32) instead of the combined output
hipError_t launch_skinny_ffn(const Fp8FfnArgs& f, const Fp8CombineArgs& c, hipStream_t s);
hipError_t launch_skinny_matmul(const Fp8MatmulArgs& a, hipStream_t s);
hipError_t launch_combine_fp8(const Fp8CombineArgs& a, hipStream_t s);

// The 16-bit hand-off of the per-pair outputs: each 64 columns of a row are fp16
// values times one power of two, the exponent of the largest.  Same bytes as
// bf16 (and 1/16 of a byte a value for the scales), an eighth of its rounding,
// and no overflow: with bf16 the rounding of the pairs was as large as that of a
// bf16 output, and its error against 64 bits 1.65 times the plain form's.
constexpr int kPairBlock = 64;

// ------------------------------------------------------------------ device helpers

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float elem_f32(__bf16 v) { return (float)v; }

// The quantiser's rule for one block: a = max|x| > 0 (finite), codes
// e4m3(x * 448 / a), scale a / 448.  x * 448 / a is formed as t / m with
// a = m * 2^e, 1 <= m < 2, t = x * (448 * 2^-e) (in range for every finite a
// >= 2^-116; a smaller a counts as 2^-116) and one residual step on the
// hardware reciprocal.  Where the quotient is an fp32 value (every tie between
// two codes for bf16 and fp16 inputs is one) the step gives it exactly:
// q0 is within 2 ulp, the residual t - q0*m is exact in an fma, and the
// correction errs by 2^-23 of those 2 ulp.  So ties resolve to even as in
// exact arithmetic.
struct Fp8Rule {
    float c, m, r, d;
    __device__ __forceinline__ explicit Fp8Rule(float amax) {
        const float a = fmaxf(amax, 0x1p-116f);
        const uint32_t b = __float_as_uint(a);
        c = __uint_as_float(((262u - (b >> 23)) << 23) | 0x600000u);   // 1.75 * 2^(8 - e)
        m = __uint_as_float((b & 0x7FFFFFu) | 0x3F800000u);
        r = __builtin_amdgcn_rcpf(m);
        d = amax > 0.0f ? __fdiv_rn(a, 448.0f) : 0.0f;
    }
    __device__ __forceinline__ float quot(float x) const {
        const float t = x * c;
        const float q0 = t * r;
        return fmaf(fmaf(-q0, m, t), r, q0);
    }
    // four values to four codes (round to nearest even; |quotient| <= 448*(1 + 2^-22), far below
    // the 464 where rounding would leave the format)
    __device__ __forceinline__ uint32_t pack4(float x0, float x1, float x2, float x3) const {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(quot(x0), quot(x1), 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(quot(x2), quot(x3), v, true);
        return (uint32_t)v;
    }
};

typedef int v8i_f8 __attribute__((ext_vector_type(8)));
typedef float v4f_f8 __attribute__((ext_vector_type(4)));
typedef _Float16 v8h_f8 __attribute__((ext_vector_type(8)));
typedef _Float16 v2h_f8 __attribute__((ext_vector_type(2)));

// Sixteen bytes of zeros: the source of copies past a row's last column.
__device__ __attribute__((aligned(16))) const uint32_t g_fp8_zero[4] = {0, 0, 0, 0};

// One asynchronous copy instruction of a wave: lane l's 16 (or
// 4) bytes at src go to LDS byte lds + 16*l (or 4*l).  lds is wave-uniform.
// The compiler does not count these loads (with its own builtin it waits for
// all of them before any LDS read, which leaves no stage in flight); the
// kernels wait on vmcnt themselves.  No output register is written, and the
// kernels hold nothing in m0.  Volatile but no memory clobber: LDS reads of
// other buffers may move past a copy, none moves past the waits and barriers.
__device__ __forceinline__ void copy16_lds(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src));
}
__device__ __forceinline__ void copy4_lds(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src));
}
__device__ __forceinline__ uint64_t wave_uniform(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | lo;
}
// The same from a wave-uniform base and a 32-bit offset per lane.
__device__ __forceinline__ void copy16_lds(uint64_t base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
                 "v"(off), "s"(wave_uniform(base)));
}
__device__ __forceinline__ void copy4_lds(uint64_t base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
                 "v"(off), "s"(wave_uniform(base)));
}
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// All of this wave's LDS reads are in registers, then the workgroup meets.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// The block product of one 16-row and one 16-token fragment: lane 16*g + r holds
// columns 16*g .. and 64 + 16*g .. (16 codes each) of row or token r, the same
// columns in both operands, so the MFMA's own column order does not matter.
template <bool EXACT>
struct Fp8Frag;

template <>
struct Fp8Frag<false> {
    v8i_f8 v;
    __device__ __forceinline__ void set(int4 a, int4 b) { v = v8i_f8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}; }
    __device__ __forceinline__ v4f_f8 times(const Fp8Frag& o) const {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, o.v, v4f_f8{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
    }
};

template <>
struct Fp8Frag<true> {
    v8h_f8 v[4];
    __device__ __forceinline__ static v8h_f8 widen(int lo, int hi) {
        const v2h_f8 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
        const v2h_f8 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
        const v2h_f8 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
        const v2h_f8 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
        return v8h_f8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    __device__ __forceinline__ void set(int4 a, int4 b) {
        v[0] = widen(a.x, a.y);
        v[1] = widen(a.z, a.w);
        v[2] = widen(b.x, b.y);
        v[3] = widen(b.z, b.w);
    }
    __device__ __forceinline__ v4f_f8 times(const Fp8Frag& o) const {
        v4f_f8 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[i], o.v[i], t, 0, 0, 0);
        return t;
    }
};

}  // namespace moe

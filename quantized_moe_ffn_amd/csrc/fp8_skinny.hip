// fp8_skinny.hip — the block-scaled products for few rows: the dense product of
// small batches, and the expert layer of decode batches.
//
// Few tokens leave a product bound by reading the weights once, and by latency:
// the tiles of fp8_gemm.hip would give too few workgroups.  Here a workgroup
// takes 16 or 32 weight rows and its eight waves split the columns block by
// block (wave w: blocks w, w + 8, ...).  A wave loads its fragments straight
// from global memory into registers, several blocks at once, with no barrier
// in the loop; the eight partial tiles meet in LDS and are added in wave order.
// The MFMA (fp8_gemm.hip) makes up to 16 tokens cost what one does.
#include "fp8.h"

namespace moe {

namespace {

constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyThreads = kSkinnyWaves * kWave;

// Adds blocks kb0, kb0 + step, ... below KB of RT row tiles x TT token tiles to
// acc.  pa/pb: this lane's row and token base (row or token r16, column 32*g of
// block 0); ws: the row tile's block scales (wave-uniform), xs: the token's.
template <bool EXACT, int RT, int TT, int NBK>
__device__ __forceinline__ void skinny_blocks(const uint8_t* const (&pa)[RT], const float* const (&ws)[RT],
                                              const uint8_t* const (&pb)[TT], const float* const (&xs)[TT], int K,
                                              int kb0, int step, v4f_f8 (&acc)[RT][TT]) {
    const int KB = (K + kFp8Block - 1) / kFp8Block;
    const int c = ((threadIdx.x & (kWave - 1)) >> 4) * 32;
    const int4 zero = make_int4(0, 0, 0, 0);
    for (int kb = kb0; kb < KB; kb += NBK * step) {
        int4 a[NBK][RT][2], b[NBK][TT][2];
        float wv[NBK][RT], xv[NBK][TT];
#pragma unroll
        for (int u = 0; u < NBK; ++u) {
            const int q = kb + u * step;
            const bool l0 = q * kFp8Block + c < K, l1 = q * kFp8Block + c + 16 < K;   // false for a whole block past K
            const int qs = min(q, KB - 1);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int4* p = reinterpret_cast<const int4*>(pa[i] + (int64_t)q * kFp8Block);
                a[u][i][0] = l0 ? p[0] : zero;
                a[u][i][1] = l1 ? p[1] : zero;
                wv[u][i] = ws[i][qs];
            }
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const int4* p = reinterpret_cast<const int4*>(pb[j] + (int64_t)q * kFp8Block);
                b[u][j][0] = l0 ? p[0] : zero;
                b[u][j][1] = l1 ? p[1] : zero;
                xv[u][j] = xs[j][qs];
            }
        }
#pragma unroll
        for (int u = 0; u < NBK; ++u) {
            Fp8Frag<EXACT> fa[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) fa[i].set(a[u][i][0], a[u][i][1]);
            const bool live = kb + u * step < KB;
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                Fp8Frag<EXACT> fb;
                fb.set(b[u][j][0], b[u][j][1]);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const v4f_f8 t = fa[i].times(fb);
                    const float s = live ? xv[u][j] * wv[u][i] : 0.0f;
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(t[v], s, acc[i][j][v]);
                }
            }
        }
    }
}

// Sum of the waves' partial tiles in wave order; part: [waves][tiles][64 lanes][4].
__device__ __forceinline__ float skinny_sum(const float* part, int tiles, int tile, int row, int tok) {
    const float* p = part + ((int64_t)tile * kWave + (row >> 2) * 16 + tok) * 4 + (row & 3);
    float s = p[0];
#pragma unroll
    for (int w = 1; w < kSkinnyWaves; ++w) s += p[(int64_t)w * tiles * kWave * 4];
    return s;
}

// ------------------------------------------------------------------ dense

template <bool EXACT, int RT, int TT, int NBK>
__global__ void __launch_bounds__(kSkinnyThreads) skinny_matmul_kernel(const Fp8MatmulArgs a, int n_rt) {
    __shared__ float s_part[kSkinnyWaves][RT * TT][kWave][4];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, g = lane >> 4;
    const int N = a.w.rows, K = a.w.cols, KB = (K + kFp8Block - 1) / kFp8Block;
    const int n0 = (blockIdx.x % n_rt) * RT * 16, t0 = (blockIdx.x / n_rt) * TT * 16;
    const uint8_t *pa[RT], *pb[TT];
    const float *ws[RT], *xs[TT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        pa[i] = a.w.data + (int64_t)min(n0 + i * 16 + r16, N - 1) * a.w.row_stride + g * 32;
        ws[i] = a.w.scale + (int64_t)(min(n0 + i * 16, N - 1) / kFp8Block) * KB;
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int64_t t = min(t0 + j * 16 + r16, a.T - 1);
        pb[j] = a.xq + t * K + g * 32;
        xs[j] = a.xs + t * KB;
    }
    v4f_f8 acc[RT][TT] = {};
    skinny_blocks<EXACT, RT, TT, NBK>(pa, ws, pb, xs, K, wave, kSkinnyWaves, acc);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) *reinterpret_cast<v4f_f8*>(s_part[wave][i * TT + j][lane]) = acc[i][j];
    __syncthreads();
    for (int o = tid; o < RT * TT * 256; o += kSkinnyThreads) {
        const int row = o % (16 * RT), tok = o / (16 * RT);
        const int n = n0 + row, t = t0 + tok;
        if (n >= N || t >= a.T) continue;
        const float s = skinny_sum(&s_part[0][0][0][0], RT * TT, (row >> 4) * TT + (tok >> 4), row & 15, tok & 15);
        const int64_t at = (int64_t)t * a.ldy + n;
        if (a.yt == ElemType::kF32)
            ((float*)a.y)[at] = s;
        else if (a.yt == ElemType::kF16)
            ((_Float16*)a.y)[at] = (_Float16)s;
        else
            ((__bf16*)a.y)[at] = (__bf16)s;
    }
}

// ------------------------------------------------------------------ layer of few pairs

// Gate/up of one (token, slot) pair, or of up to 16 tokens of the shared
// expert: 16 rows of I.  h = silu(gate) * up goes out in fp32; its quantisation
// needs all 128 rows of a block, so the down kernel's waves do it as they read.
template <bool EXACT>
__global__ void __launch_bounds__(kSkinnyThreads) skinny_gateup_kernel(const Fp8FfnArgs f, int n_it) {
    __shared__ float s_part[kSkinnyWaves][2][kWave][4];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, g = lane >> 4;
    const int P = f.T * f.k;
    const int item = blockIdx.x / n_it, i0 = (blockIdx.x - item * n_it) * 16;
    const int KB = f.H / kFp8Block;
    const bool shared = item >= P;
    Fp8Mat wg = shared ? f.sgate : f.gate, wu = shared ? f.sup : f.up;
    int n_tok = 1, t0 = shared ? (item - P) * 16 : item / f.k;
    int64_t row0 = item;
    if (shared) {
        n_tok = min(16, f.T - t0);
        row0 = P + t0;
    } else {
        const int e = f.r.idx[item];
        if ((uint32_t)e >= (uint32_t)f.E) {   // uniform over the workgroup
            if (tid == 0) raise_error(kErrExpertRange);
            return;
        }
        const int64_t ns = (int64_t)(f.I / kFp8Block) * KB;
        wg.data += e * wg.expert_stride;
        wg.scale += e * ns;
        wu.data += e * wu.expert_stride;
        wu.scale += e * ns;
    }
    const int64_t t = t0 + min(r16, n_tok - 1);
    const int64_t so = (int64_t)(i0 / kFp8Block) * KB;
    const uint8_t* const pa[2] = {wg.data + (i0 + r16) * wg.row_stride + g * 32, wu.data + (i0 + r16) * wu.row_stride + g * 32};
    const float* const ws[2] = {wg.scale + so, wu.scale + so};
    const uint8_t* const pb[1] = {f.xq + t * f.H + g * 32};
    const float* const xs[1] = {f.xs + t * KB};
    v4f_f8 acc[2][1] = {};
    skinny_blocks<EXACT, 2, 1, EXACT ? 2 : 4>(pa, ws, pb, xs, f.H, wave, kSkinnyWaves, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<v4f_f8*>(s_part[wave][i][lane]) = acc[i][0];
    __syncthreads();
    if (tid < 16 * n_tok) {
        const int row = tid & 15, tok = tid >> 4;
        const float gv = skinny_sum(&s_part[0][0][0][0], 2, 0, row, tok);
        const float uv = skinny_sum(&s_part[0][0][0][0], 2, 1, row, tok);
        f.hf[(row0 + tok) * f.I + i0 + row] = silu_f32(gv) * uv;
    }
}

// Down of one token: 16 rows of H for all its slots, wave w taking slots w,
// w + 8, ... (slot k: the shared expert).  h is quantised per 128 columns as it
// is read: lane l holds columns 2l, 2l + 1 of a block.  Four blocks at a time.
// combine: out = sum_j w_j y_j (+ s_t * shared) in slot order; else y_pair / y_shared.
template <bool EXACT>
__global__ void __launch_bounds__(kSkinnyThreads) skinny_down_kernel(const Fp8FfnArgs f, const Fp8CombineArgs c, int n_ht) {
    constexpr int kCh = 4;
    __shared__ __attribute__((aligned(16))) uint8_t s_q[kSkinnyWaves][kCh * kFp8Block];
    __shared__ float s_y[kMaxSlots][16];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, g = lane >> 4;
    const int t = blockIdx.x / n_ht, n0 = (blockIdx.x - t * n_ht) * 16;
    const int KB = f.I / kFp8Block, P = f.T * f.k;
    const int slots = f.k + (f.has_shared ? 1 : 0);
    for (int j = wave; j < slots; j += kSkinnyWaves) {
        const bool shared = j == f.k;
        Fp8Mat wd = shared ? f.sdown : f.down;
        const int64_t row = shared ? (int64_t)P + t : (int64_t)t * f.k + j;
        if (!shared) {
            const int e = f.r.idx[row];
            if ((uint32_t)e >= (uint32_t)f.E) {
                if (lane == 0) raise_error(kErrExpertRange);
                if (lane < 16) s_y[j][lane] = 0.0f;
                continue;
            }
            wd.data += e * wd.expert_stride;
            wd.scale += e * ((int64_t)(f.H / kFp8Block) * KB);
        }
        const uint8_t* pa = wd.data + (n0 + r16) * wd.row_stride + g * 32;
        const float* ws = wd.scale + (int64_t)(n0 / kFp8Block) * KB;
        const float* h = f.hf + row * f.I;
        v4f_f8 acc = {0.f, 0.f, 0.f, 0.f};
        for (int kb = 0; kb < KB; kb += kCh) {
            const int n = min(kCh, KB - kb);
            int4 a[kCh][2];
            float2 hv[kCh];
            float d[kCh], wv[kCh];
#pragma unroll
            for (int u = 0; u < kCh; ++u) {
                const int q = min(kb + u, KB - 1);
                const int4* p = reinterpret_cast<const int4*>(pa + (int64_t)q * kFp8Block);
                a[u][0] = p[0];
                a[u][1] = p[1];
                hv[u] = *reinterpret_cast<const float2*>(h + q * kFp8Block + 2 * lane);
                wv[u] = ws[q];
            }
            __builtin_amdgcn_wave_barrier();   // the reads of the last chunk's codes are done (LDS is in order per wave)
#pragma unroll
            for (int u = 0; u < kCh; ++u) {
                const uint32_t m = wave_max_u32(max(__float_as_uint(hv[u].x) & 0x7FFFFFFFu, __float_as_uint(hv[u].y) & 0x7FFFFFFFu));
                const bool fin = m < 0x7F800000u;
                if (!fin && lane == 0) raise_error(kErrActNonFinite);
                const Fp8Rule rule(__uint_as_float(fin ? m : 0u));
                const uint32_t v = fin ? rule.pack4(hv[u].x, hv[u].y, 0.f, 0.f) : 0u;
                *reinterpret_cast<uint16_t*>(&s_q[wave][u * kFp8Block + 2 * lane]) = (uint16_t)v;
                d[u] = rule.d;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int u = 0; u < kCh; ++u) {
                if (u >= n) break;
                const int4* p = reinterpret_cast<const int4*>(&s_q[wave][u * kFp8Block + g * 32]);
                Fp8Frag<EXACT> fa, fb;
                fa.set(a[u][0], a[u][1]);
                fb.set(p[0], p[1]);
                const v4f_f8 x = fa.times(fb);
                const float s = d[u] * wv[u];
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[v] = fmaf(x[v], s, acc[v]);
            }
        }
        if (r16 == 0) *reinterpret_cast<v4f_f8*>(&s_y[j][4 * g]) = acc;   // every column holds the token
    }
    __syncthreads();
    if (c.out) {
        if (tid < 16) {
            float s = 0.0f;
            for (int j = 0; j < f.k; ++j) s = fmaf(c.w[(int64_t)t * f.k + j], s_y[j][tid], s);
            if (f.has_shared) s = fmaf(c.shared_scale ? c.shared_scale[t] : 1.0f, s_y[f.k][tid], s);
            const int64_t at = (int64_t)t * f.H + n0 + tid;
            if (c.ot == ElemType::kF32)
                ((float*)c.out)[at] = s;
            else if (c.ot == ElemType::kF16)
                ((_Float16*)c.out)[at] = (_Float16)s;
            else
                ((__bf16*)c.out)[at] = (__bf16)s;
        }
    } else {
        for (int o = tid; o < slots * 16; o += kSkinnyThreads) {
            const int j = o >> 4, n = n0 + (o & 15);
            if (j == f.k)
                ((float*)f.y_shared)[(int64_t)t * f.H + n] = s_y[j][o & 15];
            else
                ((float*)f.y_pair)[((int64_t)t * f.k + j) * f.H + n] = s_y[j][o & 15];
        }
    }
}

}  // namespace

hipError_t launch_skinny_matmul(const Fp8MatmulArgs& a, hipStream_t s) {
    const bool exact = a.yt == ElemType::kF32;
    const int N = a.w.rows;
    if (a.T <= 16) {
        const int n_rt = (N + 15) / 16;
        if (exact)
            skinny_matmul_kernel<true, 1, 1, 4><<<n_rt, kSkinnyThreads, 0, s>>>(a, n_rt);
        else
            skinny_matmul_kernel<false, 1, 1, 4><<<n_rt, kSkinnyThreads, 0, s>>>(a, n_rt);
        return hipGetLastError();
    }
    const int n_rt = (N + 31) / 32;
    if (a.T <= 32) {
        if (exact)
            skinny_matmul_kernel<true, 2, 2, 2><<<n_rt, kSkinnyThreads, 0, s>>>(a, n_rt);
        else
            skinny_matmul_kernel<false, 2, 2, 4><<<n_rt, kSkinnyThreads, 0, s>>>(a, n_rt);
        return hipGetLastError();
    }
    const int n_tt = (a.T + 63) / 64;
    if (exact)
        skinny_matmul_kernel<true, 2, 4, 1><<<n_rt * n_tt, kSkinnyThreads, 0, s>>>(a, n_rt);
    else
        skinny_matmul_kernel<false, 2, 4, 2><<<n_rt * n_tt, kSkinnyThreads, 0, s>>>(a, n_rt);
    return hipGetLastError();
}

hipError_t launch_skinny_ffn(const Fp8FfnArgs& f, const Fp8CombineArgs& c, hipStream_t s) {
    const int n_it = f.I / 16, n_ht = f.H / 16;
    const int items = f.T * f.k + (f.has_shared ? (f.T + 15) / 16 : 0);
    if (f.exact) {
        skinny_gateup_kernel<true><<<items * n_it, kSkinnyThreads, 0, s>>>(f, n_it);
        skinny_down_kernel<true><<<f.T * n_ht, kSkinnyThreads, 0, s>>>(f, c, n_ht);
    } else {
        skinny_gateup_kernel<false><<<items * n_it, kSkinnyThreads, 0, s>>>(f, n_it);
        skinny_down_kernel<false><<<f.T * n_ht, kSkinnyThreads, 0, s>>>(f, c, n_ht);
    }
    return hipGetLastError();
}

}  // namespace moe

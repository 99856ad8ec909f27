// fp8_skinny.hip — the block-scaled products for few rows: the dense product of
// small batches, and the expert layer of decode batches.
//
// Few tokens leave a product bound by reading the weights once, and by latency:
// the tiles of fp8_gemm.hip would give too few workgroups.  Here a workgroup
// takes 16 weight rows (16 of gate and 16 of up) and its eight waves split the
// columns block by block (wave w: blocks w, w + 8, ...), each with a ring of
// its own in LDS that global_load_lds fills; no barrier until the eight partial
// tiles meet in LDS and are added in wave order.  Fragments loaded straight
// into registers measured 2.5 times slower: in the MFMA's layout lanes 0..15
// are 16 rows, so every quarter of a load touches 16 lines.  The copies read
// 128 contiguous bytes per eight lanes.
// The MFMA makes up to 16 tokens cost what one does.
// Measured: 16 x 2048 x 2560 3.8 us (64 x 64 tiles: 10.1); the layer of one token
// (256 experts / top-8, H 2048, I 512) 17.4 us, with the grouped tiles 39.6;
// of eight tokens, 64 pairs, 50 and 57.
#include "fp8.h"

namespace moe {

namespace {

constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyThreads = kSkinnyWaves * kWave;
constexpr int kSkinnyChunk = 8;   // blocks of a wave whose tokens' scales (and a single token's codes) are copied together

// One wave's part of a product: RT row tiles x TT token tiles of 16, over its
// blocks kb0, kb0 + step, ...  TT = 0: a single token, whose codes every MFMA
// column holds (its 128 bytes a block are copied once for eight blocks).
template <bool EXACT, int RT, int TT, int S>
struct SkinnyWave {
    static constexpr int kTiles = RT + TT;
    static constexpr int kCopies = 2 * kTiles;            // copies of one ring stage
    static constexpr int kRing = S * kTiles * 2048;
    static constexpr int kCodes = TT == 0 ? kSkinnyChunk * kFp8Block : 0;
    static constexpr int kScaleArea = 256 + 16 * TT * kSkinnyChunk * 4;   // the rows', then the tokens'
    static constexpr int kLds = kRing + kCodes + kScaleArea;   // bytes of LDS of a wave
    static constexpr int TA = TT == 0 ? 1 : TT;
    static_assert(RT + (TT == 0 ? 1 : 0) <= 8, "one copy instruction holds the rows' scales");
    static_assert(RT * (TT == 0 ? 1 : TT) * 1024 <= kRing, "the partial tiles fit the ring");

    const uint8_t* pr[RT][2];   // row operand: copy c's source (row 8c + lane/8, swizzled chunk) in block 0
    const uint8_t* pt[TA][2];   // token operand, the same; TT = 0: pt[0][0] the token's codes
    const float* ws[RT];        // block scales of the row tiles (wave-uniform)
    const float* xs[TA];        // scales of token (lane & 15) of tile j; TT = 0: the token's
    int ca;                     // first column of this lane's chunk within a block

    __device__ __forceinline__ static int chunk_col() {
        const int lane = threadIdx.x & (kWave - 1);
        return ((lane & 7) ^ (lane >> 3)) * 16;
    }

    // acc += the wave's blocks; lds: this wave's kLds bytes, l0: their LDS address
    __device__ __forceinline__ void run(const unsigned char* lds, uint32_t l0, int K, int kb0, int step,
                                        v4f_f8 (&acc)[RT][TA]) const {
        const int lane = threadIdx.x & (kWave - 1), r16 = lane & 15, g = lane >> 4;
        const int KB = (K + kFp8Block - 1) / kFp8Block;
        const int n = kb0 < KB ? (KB - 1 - kb0) / step + 1 : 0;   // blocks of this wave
        const int c0 = (g ^ (r16 & 7)) * 16, c1 = c0 ^ 64;
        const uintptr_t z = (uintptr_t)g_fp8_zero;
        auto issue = [&](int u) {
            const int kb = kb0 + u * step;
            const uint32_t st = l0 + (u % S) * kTiles * 2048;
            const bool live = kb * kFp8Block + ca < K;   // chunks past the last column read zeros
            const int64_t o = (int64_t)kb * kFp8Block;
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    copy16_lds((const void*)(live ? (uintptr_t)(pr[i][h] + o) : z), st + i * 2048 + h * 1024);
#pragma unroll
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    copy16_lds((const void*)(live ? (uintptr_t)(pt[j][h] + o) : z), st + (RT + j) * 2048 + h * 1024);
        };
        const uint32_t lx = l0 + kRing, ls = lx + kCodes;
        const unsigned char* px = lds + kRing;
        const float* ps = reinterpret_cast<const float*>(lds + kRing + kCodes);
        for (int u0 = 0; u0 < n; u0 += kSkinnyChunk) {
            const int m = min(kSkinnyChunk, n - u0);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the last chunk's reads are done
            // scales: entry q*8 + u of row tile q, then of the single token; from byte 256 [tile][block][16 tokens]
            {
                const int q = lane >> 3, kb = kb0 + (u0 + min(lane & 7, m - 1)) * step;
                const float* p = ws[0];
#pragma unroll
                for (int i = 1; i < RT; ++i) p = q == i ? ws[i] : p;
                if (TT == 0) p = q == RT ? xs[0] : p;
                copy4_lds(p + kb, ls);
            }
            if constexpr (TT == 0) {   // eight blocks of 128 codes: lanes 8u .. 8u + 7 copy block u
                const int kb = kb0 + (u0 + min(lane >> 3, m - 1)) * step, col = kb * kFp8Block + (lane & 7) * 16;
                copy16_lds((const void*)(col < K ? (uintptr_t)(pt[0][0] + col) : z), lx);
            } else {
#pragma unroll
                for (int j = 0; j < TT; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // four blocks of 16 tokens
                        const int kb = kb0 + (u0 + min(4 * h + g, m - 1)) * step;
                        copy4_lds(xs[j] + kb, ls + 256 + (j * 2 + h) * kWave * 4);
                    }
            }
#pragma unroll
            for (int u = 0; u < S; ++u)
                if (u < m) issue(u0 + u);
            for (int u = 0; u < m; ++u) {
                const int newer = min(S - 1, m - 1 - u);   // stages issued after this one
                if (newer == 0)
                    wait_vm<0>();
                else if (S == 2 || newer == 1)
                    wait_vm<kCopies>();
                else if (S == 3 || newer == 2)
                    wait_vm<2 * kCopies>();
                else
                    wait_vm<3 * kCopies>();
                const unsigned char* st = lds + ((u0 + u) % S) * kTiles * 2048 + r16 * 128;
                Fp8Frag<EXACT> fa[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    fa[i].set(*reinterpret_cast<const int4*>(st + i * 2048 + c0), *reinterpret_cast<const int4*>(st + i * 2048 + c1));
#pragma unroll
                for (int j = 0; j < TA; ++j) {
                    Fp8Frag<EXACT> fb;
                    float x;
                    if constexpr (TT == 0) {
                        const int4* p = reinterpret_cast<const int4*>(px + u * kFp8Block + g * 16);
                        fb.set(p[0], p[4]);
                        x = ps[RT * kSkinnyChunk + u];
                    } else {
                        const unsigned char* p = st + (RT + j) * 2048;
                        fb.set(*reinterpret_cast<const int4*>(p + c0), *reinterpret_cast<const int4*>(p + c1));
                        x = ps[kWave + (j * 2 + (u >> 2)) * kWave + (u & 3) * 16 + r16];
                    }
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const v4f_f8 t = fa[i].times(fb);
                        const float s = x * ps[i * kSkinnyChunk + u];
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(t[v], s, acc[i][j][v]);
                    }
                }
                if (u + S < m) {
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    issue(u0 + u + S);
                }
            }
        }
    }
};

// Sum of the waves' partial tiles in wave order; a wave leaves them as
// [tile][64 lanes][4] at the start of its LDS, `stride` bytes after the last wave's.
__device__ __forceinline__ float skinny_sum(const unsigned char* lds, int stride, int tile, int row, int tok) {
    const unsigned char* p = lds + ((tile * kWave + (row >> 2) * 16 + tok) * 4 + (row & 3)) * 4;
    float s = *reinterpret_cast<const float*>(p);
#pragma unroll
    for (int w = 1; w < kSkinnyWaves; ++w) s += *reinterpret_cast<const float*>(p + w * stride);
    return s;
}

// ------------------------------------------------------------------ dense

template <bool EXACT, int TT, int S>
__global__ void __launch_bounds__(kSkinnyThreads) skinny_matmul_kernel(const Fp8MatmulArgs a, int n_rt) {
    using W = SkinnyWave<EXACT, 1, TT, S>;
    constexpr int RT = 1, TA = W::TA;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int N = a.w.rows, K = a.w.cols, KB = (K + kFp8Block - 1) / kFp8Block;
    const int n0 = (blockIdx.x % n_rt) * 16, t0 = (blockIdx.x / n_rt) * TA * 16;
    W w;
    w.ca = W::chunk_col();
#pragma unroll
    for (int h = 0; h < 2; ++h) w.pr[0][h] = a.w.data + (int64_t)min(n0 + 8 * h + (lane >> 3), N - 1) * a.w.row_stride + w.ca;
    w.ws[0] = a.w.scale + (int64_t)(n0 / kFp8Block) * KB;
    if constexpr (TT == 0) {
        w.pt[0][0] = a.xq + (int64_t)t0 * K;
        w.xs[0] = a.xs + (int64_t)t0 * KB;
    } else {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w.pt[j][h] = a.xq + (int64_t)min(t0 + j * 16 + 8 * h + (lane >> 3), a.T - 1) * K + w.ca;
            w.xs[j] = a.xs + (int64_t)min(t0 + j * 16 + (lane & 15), a.T - 1) * KB;
        }
    }
    v4f_f8 acc[RT][TA] = {};
    w.run(lds + wave * W::kLds, lds_address(lds) + wave * W::kLds, K, wave, kSkinnyWaves, acc);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TA; ++j) *reinterpret_cast<v4f_f8*>(lds + wave * W::kLds + ((i * TA + j) * kWave + lane) * 16) = acc[i][j];
    __syncthreads();
    for (int o = tid; o < TA * 256; o += kSkinnyThreads) {
        const int row = o % 16, tok = o / 16;
        const int n = n0 + row, t = t0 + tok;
        if (n >= N || t >= a.T || (TT == 0 && tok > 0)) continue;
        const float s = skinny_sum(lds, W::kLds, tok >> 4, row, tok & 15);
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

// Gate/up of one (token, slot) pair, or of one token of the shared expert: 16
// rows of I.  h = silu(gate) * up goes out in fp32; its quantisation needs all
// 128 rows of a block, so the down kernel's waves do it as they read.
template <bool EXACT>
__global__ void __launch_bounds__(kSkinnyThreads) skinny_gateup_kernel(const Fp8FfnArgs f, int n_it) {
    using W = SkinnyWave<EXACT, 2, 0, 2>;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int P = f.T * f.k;
    const int item = blockIdx.x / n_it, i0 = (blockIdx.x - item * n_it) * 16;   // h row `item`
    const int KB = f.H / kFp8Block;
    const bool shared = item >= P;
    Fp8Mat wg = shared ? f.sgate : f.gate, wu = shared ? f.sup : f.up;
    const int t = shared ? item - P : item / f.k;
    if (!shared) {
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
    W w;
    w.ca = W::chunk_col();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t row = i0 + 8 * h + (lane >> 3);
        w.pr[0][h] = wg.data + row * wg.row_stride + w.ca;
        w.pr[1][h] = wu.data + row * wu.row_stride + w.ca;
    }
    const int64_t so = (int64_t)(i0 / kFp8Block) * KB;
    w.ws[0] = wg.scale + so;
    w.ws[1] = wu.scale + so;
    w.pt[0][0] = f.xq + (int64_t)t * f.H;
    w.xs[0] = f.xs + (int64_t)t * KB;
    v4f_f8 acc[2][1] = {};
    w.run(lds + wave * W::kLds, lds_address(lds) + wave * W::kLds, f.H, wave, kSkinnyWaves, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<v4f_f8*>(lds + wave * W::kLds + (i * kWave + lane) * 16) = acc[i][0];
    __syncthreads();
    if (tid < 16) {
        const float gv = skinny_sum(lds, W::kLds, 0, tid, 0);
        const float uv = skinny_sum(lds, W::kLds, 1, tid, 0);
        f.hf[(int64_t)item * f.I + i0 + tid] = silu_f32(gv) * uv;
    }
}

// Down of one token: 16 rows of H for all its slots, wave w taking slots w,
// w + 8, ... (slot k: the shared expert).  h is quantised per 128 columns as it
// is read: lane l holds columns 2l, 2l + 1 of a block.  Four blocks at a time.
// c.out: out = sum_j w_j y_j (+ s_t * shared) in slot order; else y_pair / y_shared.
template <bool EXACT>
__global__ void __launch_bounds__(kSkinnyThreads) skinny_down_kernel(const Fp8FfnArgs f, const Fp8CombineArgs c, int n_ht) {
    constexpr int kCh = 4;
    __shared__ __attribute__((aligned(16))) unsigned char s_w[kSkinnyWaves][kCh * 2048];
    __shared__ __attribute__((aligned(16))) uint8_t s_q[kSkinnyWaves][kCh * kFp8Block];
    __shared__ float s_y[kMaxSlots][16], s_wt[kMaxSlots];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, g = lane >> 4;
    const int t = blockIdx.x / n_ht, n0 = (blockIdx.x - t * n_ht) * 16;
    const int KB = f.I / kFp8Block, P = f.T * f.k;
    const int slots = f.k + (f.has_shared ? 1 : 0);
    const int ca = ((lane & 7) ^ (lane >> 3)) * 16;
    const int c0 = (g ^ (r16 & 7)) * 16, c1 = c0 ^ 64;
    const uint32_t l0 = lds_address(s_w[wave]);
    if (c.out && tid < slots)   // the combine's weights, fetched beside the rows
        s_wt[tid] = tid < f.k ? c.w[(int64_t)t * f.k + tid] : (c.shared_scale ? c.shared_scale[t] : 1.0f);
    for (int j = wave; j < slots; j += kSkinnyWaves) {
        const bool shared = j == f.k;
        Fp8Mat wd = shared ? f.sdown : f.down;
        const int64_t row = shared ? (int64_t)P + t : (int64_t)t * f.k + j;
        if (!shared) {
            const int e = __builtin_amdgcn_readfirstlane(f.r.idx[row]);
            if ((uint32_t)e >= (uint32_t)f.E) {
                if (lane == 0) raise_error(kErrExpertRange);
                if (lane < 16) s_y[j][lane] = 0.0f;
                continue;
            }
            wd.data += e * wd.expert_stride;
            wd.scale += e * ((int64_t)(f.H / kFp8Block) * KB);
        }
        const uint8_t* pa = wd.data + (int64_t)(n0 + (lane >> 3)) * wd.row_stride + ca;
        const float* ws = wd.scale + (int64_t)(n0 / kFp8Block) * KB;
        const float* h = f.hf + row * f.I;
        v4f_f8 acc = {0.f, 0.f, 0.f, 0.f};
        for (int kb = 0; kb < KB; kb += kCh) {
            const int n = min(kCh, KB - kb);
            float2 hv[kCh];
            float d[kCh], wv[kCh];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the last chunk's reads are done
#pragma unroll
            for (int u = 0; u < kCh; ++u) {
                if (u < n) {
                    copy16_lds(pa + (kb + u) * kFp8Block, l0 + u * 2048);
                    copy16_lds(pa + 8 * wd.row_stride + (kb + u) * kFp8Block, l0 + u * 2048 + 1024);
                }
            }
#pragma unroll
            for (int u = 0; u < kCh; ++u) {
                const int q = min(kb + u, KB - 1);
                hv[u] = *reinterpret_cast<const float2*>(h + q * kFp8Block + 2 * lane);
                wv[u] = ws[q];
            }
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
            wait_vm<0>();
#pragma unroll
            for (int u = 0; u < kCh; ++u) {
                if (u >= n) break;
                const int4* p = reinterpret_cast<const int4*>(&s_q[wave][u * kFp8Block + g * 16]);
                const unsigned char* a = s_w[wave] + u * 2048 + r16 * 128;
                Fp8Frag<EXACT> fa, fb;
                fa.set(*reinterpret_cast<const int4*>(a + c0), *reinterpret_cast<const int4*>(a + c1));
                fb.set(p[0], p[4]);
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
            for (int j = 0; j < slots; ++j) s = fmaf(s_wt[j], s_y[j][tid], s);
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

template <bool EXACT, int TT, int S>
hipError_t launch_skinny_matmul_t(const Fp8MatmulArgs& a, hipStream_t s) {
    using W = SkinnyWave<EXACT, 1, TT, S>;
    const int n_rt = (a.w.rows + 15) / 16, n_tt = (a.T + W::TA * 16 - 1) / (W::TA * 16);
    skinny_matmul_kernel<EXACT, TT, S><<<n_rt * n_tt, kSkinnyThreads, kSkinnyWaves * W::kLds, s>>>(a, n_rt);
    return hipGetLastError();
}

hipError_t launch_skinny_matmul(const Fp8MatmulArgs& a, hipStream_t s) {
    // up to 32 tokens the weights bound the product and the wider sums cost nothing
    if (a.T == 1) return launch_skinny_matmul_t<true, 0, 3>(a, s);
    if (a.T <= 16) return launch_skinny_matmul_t<true, 1, 2>(a, s);
    return launch_skinny_matmul_t<true, 2, 2>(a, s);
}

hipError_t launch_skinny_ffn(const Fp8FfnArgs& f, const Fp8CombineArgs& c, hipStream_t s) {
    using W = SkinnyWave<true, 2, 0, 2>;
    const int n_it = f.I / 16, n_ht = f.H / 16;
    const int items = f.T * f.k + (f.has_shared ? f.T : 0);
    skinny_gateup_kernel<true><<<items * n_it, kSkinnyThreads, kSkinnyWaves * W::kLds, s>>>(f, n_it);
    skinny_down_kernel<true><<<f.T * n_ht, kSkinnyThreads, 0, s>>>(f, c, n_ht);
    return hipGetLastError();
}

}  // namespace moe

// fp8_stream.hip — the grouped products of the expert layer as persistent
// workgroups: one pipeline of copies and MFMAs runs through all the tiles of a
// workgroup.
//
// The tiles of fp8_gemm.hip start cold: the list entry, the bucket, the pair ids
// and the first copies are a chain of memory latencies, about 7 us against the
// 4 to 16 us a tile's blocks take (down: 11.5 us a tile for four blocks; gate/up
// of 4,096 tokens 212 us where the weights' 537 MB need about 100).  Here a
// workgroup takes items j, j + step, ... of its XCD's contiguous part of the
// list (item: 256 weight rows x one token tile; the row blocks of a tile are
// neighbours, so workgroups that run at once share tokens and weights in L2),
// and the copies run STAGES - 1 blocks ahead across item borders.  An item's
// pair ids and weight scales are copied to LDS one item ahead, its list entry
// two, so that the main loop holds no load the compiler would wait for (its
// wait would drain the copies too).
//
// What it takes (4,096 tokens of 256 experts / top-8, H 2048, I 512 of bf16):
// gate/up 158 us, down 104 us, against about 85 and 65 us of weights, tokens
// and results at 6.5 TB/s, what streaming reads reach.  With the copies left out gate/up took
// 160 us, with copies and MFMAs left out 145 us, with LDS reads and MFMAs left
// out 150 us: no unit is busy throughout; the rest is the items' ends
// (SiLU, requantisation, stores), one barrier a block and the ragged last items.
// Tried and left out: two groups of waves alternating LDS reads and MFMAs as in
// the dense tiles, reading token fragments one tile ahead, evening out the
// workgroups' tokens by the order of the list (no gain), prefetching the next
// item's weights into L2 (slower).
//
// Needs K a multiple of 512 (token scales are copied four blocks at a time),
// 16-byte aligned token scales and at most 8,192 (the 64 weight scales of an
// item are one copy).
#include "fp8.h"

namespace moe {

namespace {

constexpr int kStreamMaxK = 64 * kFp8Block;

// One work item (row block nb of list entry e, m0, n_tok, row0), the same in every lane.
struct StreamItem {
    int e, nb, mt0, n_tok, row0;
    bool shared;
};

template <int NWN, int NWM, int WN, int WM, int STAGES>
struct StreamShape {
    static constexpr int kWaves = NWN * NWM, kThreads = kWaves * kWave;
    static constexpr int NR = NWN * WN * 16, MT = NWM * WM * 16;
    static constexpr int NA = NR / 8 / kWaves, NB = MT / 8 / kWaves;
    static constexpr int kLoads = NA + NB;            // copies of a wave in every stage
    static constexpr int kSegs = MT < 64 ? 1 : MT / 64;
    static constexpr int kTok = kSegs * 64;
    static constexpr int kStage = (NR + MT) * 128, kRing = STAGES * kStage;
    static constexpr int kXs = kTok * 16;             // token scales: [token][4 blocks], two buffers
    static constexpr int kMeta = kTok * 4 + 512;      // an item's pair ids and 2 x 64 weight scales, three buffers
    static constexpr int kEntry = kRing + 2 * kXs + 3 * kMeta;   // list entries: 64 words each (a copy's size), two buffers
    static constexpr int kLds = kEntry + 512;
    static_assert(NA * 8 * kWaves == NR && NB * 8 * kWaves == MT && NR == 256, "copies divide evenly");
    static_assert(kWaves >= kSegs + 2 && kLds + NWN * MT * 4 <= 160 * 1024 && STAGES <= 4, "shape");
};

template <int MODE, bool EXACT, int NWN, int NWM, int WN, int WM, int STAGES>
__global__ void __launch_bounds__(NWN* NWM* kWave) fp8_stream_kernel(const Fp8TileArgs a) {
    using C = StreamShape<NWN, NWM, WN, WM, STAGES>;
    constexpr bool kGu = MODE == kFp8GateUp;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ uint32_t s_amax[kGu ? NWN : 1][C::MT];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wn = wave % NWN, wm = wave / NWN;
    const int g = lane >> 4, r16 = lane & 15;
    const int K = a.K, KB = K / kFp8Block, P = a.T * a.k;
    const uint32_t lds0 = lds_address(lds);

    const int n_work = __builtin_amdgcn_readfirstlane(*a.tl.n_items) * a.nblocks;
    const int chunk = (n_work + 7) / 8, step = gridDim.x / 8;
    const int first = (blockIdx.x % 8) * chunk + blockIdx.x / 8;
    const int lim = min((int)(blockIdx.x % 8 + 1) * chunk, n_work);
    if (first >= lim) return;
    const int total = ((lim - first - 1) / step + 1) * KB;   // stages of this workgroup

    // Copies item w's list entry into buffer b (wave 0); reads the one copied there.
    auto fetch_entry = [&](int w, int b) {
        if (wave == 0) copy4_lds((uint64_t)(a.tl.items + w / a.nblocks), (uint32_t)(lane & 3) * 4, lds0 + C::kEntry + b * 256);
    };
    auto read_entry = [&](int w, int b) {
        const int4 v = *reinterpret_cast<const int4*>(lds + C::kEntry + b * 256);
        StreamItem it;
        it.nb = w % a.nblocks;
        it.e = __builtin_amdgcn_readfirstlane(v.x);
        it.mt0 = __builtin_amdgcn_readfirstlane(v.y);
        it.n_tok = __builtin_amdgcn_readfirstlane(v.z);
        it.row0 = __builtin_amdgcn_readfirstlane(v.w);
        it.shared = it.e >= a.E;
        return it;
    };
    // Copies of an item's pair ids and weight scales into buffer b.
    auto fetch_meta = [&](const StreamItem& it, int b) {
        const uint32_t at = lds0 + C::kRing + 2 * C::kXs + b * C::kMeta;
        if (wave < C::kSegs) {
            const int m = min(wave * 64 + lane, it.n_tok - 1);
            if (!it.shared)
                copy4_lds((uint64_t)(a.pair + it.row0), (uint32_t)m * 4, at + wave * 256);
        } else if (wave < C::kSegs + 2) {
            const int q = wave - C::kSegs;
            const int sb = kGu ? it.nb : min(2 * it.nb + q, (a.N - 1) / kFp8Block);
            const float* sc = kGu && q ? (it.shared ? a.s1.scale : a.w1.scale) : (it.shared ? a.s0.scale : a.w0.scale);
            const int64_t rb = it.shared ? 0 : (int64_t)it.e * ((a.N + kFp8Block - 1) / kFp8Block);
            copy4_lds((uint64_t)(sc + (rb + sb) * KB), (uint32_t)min(lane, KB - 1) * 4,
                      at + C::kTok * 4 + q * 256);
        }
    };

    // The item whose blocks are being copied: 32-bit offsets from wave-uniform bases.
    const int lr = lane >> 3, ca = ((lane & 7) ^ lr) * 16;
    uint64_t ba[C::NA], bb = 0, bs = 0;
    uint32_t oa[C::NA], ob[C::NB], os = 0;
    auto setup = [&](const StreamItem& it, int b) {
        const int* pr = reinterpret_cast<const int*>(lds + C::kRing + 2 * C::kXs + b * C::kMeta);
        const uint8_t* d0 = it.shared ? a.s0.data : a.w0.data + (int64_t)it.e * a.w0.expert_stride;
        const uint8_t* d1 = !kGu ? d0 : (it.shared ? a.s1.data : a.w1.data + (int64_t)it.e * a.w1.expert_stride);
        const int r0 = (int)(it.shared ? a.s0.row_stride : a.w0.row_stride);
        const int r1 = !kGu ? r0 : (int)(it.shared ? a.s1.row_stride : a.w1.row_stride);
#pragma unroll
        for (int i = 0; i < C::NA; ++i) {
            const int R8 = (wave + i * C::kWaves) * 8;
            if constexpr (kGu) {
                const int w_ = R8 / (WN * 16), r_ = R8 % (WN * 16);
                const int row = it.nb * (C::NR / 2) + w_ * (WN / 2 * 16) + pair_row(r_ % (WN / 2 * 16));
                const bool up = r_ >= WN / 2 * 16;
                ba[i] = wave_uniform((uint64_t)(up ? d1 : d0) + (uint64_t)row * (uint32_t)(up ? r1 : r0));
                oa[i] = (uint32_t)(pair_row(lr) * (up ? r1 : r0) + ca);
            } else {
                const int row0 = it.nb * C::NR;
                ba[i] = wave_uniform((uint64_t)d0 + (uint64_t)row0 * (uint32_t)r0);
                oa[i] = (uint32_t)((min(row0 + pair_row(R8 + lr), a.N - 1) - row0) * r0 + ca);
            }
        }
        // token operand: gate/up gathers rows of x, down reads the bucket's rows of h
        const int last = it.n_tok - 1;
        auto src = [&](int m) -> uint32_t {
            m = min(m, last);
            if constexpr (!kGu) return m;
            if (it.shared) return it.mt0 + m;
            const uint32_t p = pr[m];
            if (p >= (uint32_t)P) raise_error(kErrPairRange);
            return p < (uint32_t)P ? p / (uint32_t)a.k : 0u;
        };
        const int64_t tok0 = kGu ? 0 : it.row0;
        bb = wave_uniform((uint64_t)(a.xq + tok0 * K));
        bs = wave_uniform((uint64_t)(a.xs + tok0 * KB));
#pragma unroll
        for (int i = 0; i < C::NB; ++i) ob[i] = src((wave + i * C::kWaves) * 8 + lr) * (uint32_t)K + ca;
        os = src(min(wave, C::kSegs - 1) * 64 + lane) * (uint32_t)KB * 4;
    };

    int iw = first, ikb = 0, islot = 0, ixs = 0, ibuf = 0, ient = 0;   // the copies' item, block, ring slot and buffers
    fetch_entry(first, 0);
    fetch_entry(min(first + step, lim - 1), 1);
    wait_vm<0>();
    lds_barrier();
    StreamItem cur = read_entry(first, 0), nxt = read_entry(min(first + step, lim - 1), 1);
    fetch_meta(cur, 0);
    wait_vm<0>();
    lds_barrier();
    setup(cur, 0);
    if (first + step < lim) {
        fetch_meta(nxt, 1);
        if (first + 2 * step < lim) fetch_entry(first + 2 * step, 0);
    }
    // Copy c of the next block (kLoads of them, then possibly the token scales).  They go out between the
    // MFMAs: the address unit takes about 16 cycles for each, 768 a block, which would otherwise stand
    // between the barrier and the first LDS reads.
    auto copy = [&](int c) {
        const uint32_t la = lds0 + islot * C::kStage + wave * 1024;
        const uint64_t o = (uint64_t)ikb * kFp8Block;
        if (c < C::NA)
            copy16_lds(ba[c < C::NA ? c : 0] + o, oa[c < C::NA ? c : 0], la + c * C::kWaves * 1024);
        else
            copy16_lds(bb + o, ob[c < C::NA ? 0 : c - C::NA], la + C::NR * 128 + (c - C::NA) * C::kWaves * 1024);
    };
    // After the copies: moves on to the next block; past an item's last one to the next item, whose pair ids
    // (and the entry after it) were copied a whole item ago (K/128 > STAGES blocks: older than the block just
    // waited for).
    auto advance = [&]() {
        if ((ikb & 3) == 0) {
            if (wave < C::kSegs) copy16_lds(wave_uniform(bs + 4 * (uint64_t)ikb), os, lds0 + C::kRing + ixs * C::kXs + wave * 1024);
            ixs ^= 1;
        }
        islot = islot + 1 == STAGES ? 0 : islot + 1;
        if (++ikb == KB) {
            ikb = 0;
            iw += step;
            if (iw < lim) {
                ibuf = ibuf == 2 ? 0 : ibuf + 1;
                cur = nxt;
                setup(cur, ibuf);
                if (iw + step < lim) {
                    nxt = read_entry(iw + step, ient);
                    ient ^= 1;
                    fetch_meta(nxt, ibuf == 2 ? 0 : ibuf + 1);
                    if (iw + 2 * step < lim) fetch_entry(iw + 2 * step, ient);
                }
            }
        }
    };

    // the item being computed
    StreamItem ci = cur;
    int cbuf = 0, kb = 0, st = 0, xs = 0;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {   // an item has at least STAGES blocks
#pragma unroll
        for (int c = 0; c < C::kLoads; ++c) copy(c);
        advance();
    }

    const int c0 = (g ^ (r16 & 7)) * 16, c1 = c0 ^ 64;
    const unsigned char* la0 = lds + (wn * WN * 16 + r16) * 128 + c0;
    const unsigned char* la1 = lds + (wn * WN * 16 + r16) * 128 + c1;
    // a wave's token tile j is the item's tile j * NWM + wm, so that a part-filled item loads the waves alike;
    // tiles past the item's last token are skipped (at 4,096 tokens a third of them)
    auto tok = [&](int j) { return (j * NWM + wm) * 16 + r16; };
    const unsigned char* lb0 = lds + C::NR * 128 + tok(0) * 128 + c0;
    const unsigned char* lb1 = lds + C::NR * 128 + tok(0) * 128 + c1;
    const unsigned char* lsx = lds + C::kRing + tok(0) * 16;
    v4f_f8 acc[WN][WM] = {};
    int here = 0;   // blocks from s on whose copies were waited for before an epilogue's stores
    for (int s = 0; s < total; ++s) {
        if (here > 0)
            --here;
        else if (s + STAGES - 2 < total)
            wait_vm<(STAGES - 2) * C::kLoads>();
        else
            wait_vm<0>();
        lds_barrier();
        const bool more = s + STAGES - 1 < total;
        const float* pw = reinterpret_cast<const float*>(lds + C::kRing + 2 * C::kXs + cbuf * C::kMeta + C::kTok * 4);
        // down: 256 rows are two scale blocks, four waves of 64 rows
        const float wb0 = pw[(kGu ? 0 : (wn >> 1) * 64) + kb], wb1 = kGu ? pw[64 + kb] : 0.f;
        const int nj = (ci.n_tok + 15) / 16 - wm;   // token tiles j * NWM + wm of this wave
        Fp8Frag<EXACT> fa[WN];
#pragma unroll
        for (int i = 0; i < WN; ++i)
            fa[i].set(*reinterpret_cast<const int4*>(la0 + st + i * 2048), *reinterpret_cast<const int4*>(la1 + st + i * 2048));
#pragma unroll
        for (int j = 0; j < WM; ++j) {
            if (j * NWM < nj) {
                Fp8Frag<EXACT> fb;
                fb.set(*reinterpret_cast<const int4*>(lb0 + st + j * NWM * 2048),
                       *reinterpret_cast<const int4*>(lb1 + st + j * NWM * 2048));
                const float x = *reinterpret_cast<const float*>(lsx + xs + j * NWM * 256 + (kb & 3) * 4);
                const float s0 = x * wb0, s1 = kGu ? x * wb1 : 0.f;
#pragma unroll
                for (int i = 0; i < WN; ++i) {
                    const v4f_f8 t = fa[i].times(fb);
                    const float sc = kGu && i >= WN / 2 ? s1 : s0;
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(t[v], sc, acc[i][j][v]);
                }
            }
            if (more) {
#pragma unroll
                for (int c = C::kLoads * j / WM; c < C::kLoads * (j + 1) / WM; ++c) copy(c);
            }
        }
        if (more) advance();
        st = st + C::kStage == C::kRing ? 0 : st + C::kStage;
        if ((kb & 3) == 3) xs ^= C::kXs;
        if (++kb < KB) continue;

        // The item's results: value v of acc[i][j] is weight row pair_col(i, g) + v of the wave, token tok(j).
        // The copies of the next item's first blocks are in flight.
        if constexpr (kGu) {
            constexpr int HI = WN / 2;
#pragma unroll
            for (int j = 0; j < WM; ++j) {
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < HI; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float h = silu_f32(acc[i][j][v]) * acc[i + HI][j][v];
                        acc[i][j][v] = h;
                        mx = max(mx, __float_as_uint(h) & 0x7FFFFFFFu);
                    }
                mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, kWave));
                mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, kWave));
                if (g == 0) s_amax[wn][tok(j)] = mx;
            }
            wait_vm<0>();
            here = STAGES - 1;
            lds_barrier();
            const int64_t row0 = ci.row0;
#pragma unroll
            for (int j = 0; j < WM; ++j) {
                const int m = tok(j);
                uint32_t mx = s_amax[0][m];
#pragma unroll
                for (int q = 1; q < NWN; ++q) mx = max(mx, s_amax[q][m]);
                const bool fin = mx < 0x7F800000u;
                if (m >= ci.n_tok) continue;
                if (!fin) raise_error(kErrActNonFinite);
                const Fp8Rule rule(__uint_as_float(fin ? mx : 0u));
#pragma unroll
                for (int i = 0; i < HI; i += 2) {
                    const uint32_t q0 = fin ? rule.pack4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]) : 0u;
                    const uint32_t q1 =
                        fin ? rule.pack4(acc[i + 1][j][0], acc[i + 1][j][1], acc[i + 1][j][2], acc[i + 1][j][3]) : 0u;
                    const int col = ci.nb * (C::NR / 2) + wn * HI * 16 + pair_col(i, g);
                    *reinterpret_cast<uint2*>(a.hq + (row0 + m) * a.N + col) = make_uint2(q0, q1);
                }
                if (wn == 0 && g == 0) a.hs[(row0 + m) * (a.N / kFp8Block) + ci.nb] = rule.d;
            }
        } else {
            const int* pr = reinterpret_cast<const int*>(lds + C::kRing + 2 * C::kXs + cbuf * C::kMeta);
            void* base = ci.shared ? a.y_shared : a.y_pair;
            float* scale = a.y_scale + (ci.shared ? (int64_t)P * (a.N / kPairBlock) : 0);
            wait_vm<0>();
            here = STAGES - 1;
#pragma unroll
            for (int j = 0; j < WM; ++j) {
                const int m = tok(j);
                int row = ci.shared ? ci.mt0 + m : pr[m];
                if (m >= ci.n_tok) {
                    row = -1;
                } else if (!ci.shared && (uint32_t)row >= (uint32_t)P) {
                    raise_error(kErrPairRange);
                    row = -1;
                }
                v4f_f8 y[WN];
#pragma unroll
                for (int i = 0; i < WN; ++i) y[i] = acc[i][j];
                store_row64<WN>(y, base, scale, a.pair16, row, ci.nb * C::NR + wn * WN * 16, a.N);
            }
        }
#pragma unroll
        for (int i = 0; i < WN; ++i)
#pragma unroll
            for (int j = 0; j < WM; ++j) acc[i][j] = v4f_f8{0.f, 0.f, 0.f, 0.f};
        kb = 0;
        ci = cur;   // the copies are STAGES - 1 blocks ahead: in the next item
        cbuf = cbuf == 2 ? 0 : cbuf + 1;
    }
}

constexpr int kCus = 256;

template <int MODE, bool EXACT, int NWN, int NWM, int WN, int WM, int STAGES>
hipError_t launch_stream(const Fp8TileArgs& a, int64_t n_work, hipStream_t s) {
    using C = StreamShape<NWN, NWM, WN, WM, STAGES>;
    const int64_t per_cu = (C::kLds + NWN * C::MT * 4) * 2 <= 160 * 1024 ? 2 : 1;
    const int64_t want = (n_work + 7) / 8 * 8;
    const unsigned grid = (unsigned)(want < per_cu * kCus ? want : per_cu * kCus);
    fp8_stream_kernel<MODE, EXACT, NWN, NWM, WN, WM, STAGES><<<grid, C::kThreads, C::kLds, s>>>(a);
    return hipGetLastError();
}

}  // namespace

}  // namespace moe

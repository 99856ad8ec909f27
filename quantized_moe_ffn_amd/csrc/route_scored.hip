// route_scored.hip — expert selection from router logits by a score rule:
// softmax or sigmoid scores, a per-expert balance bias, group-limited top-k,
// renormalised and scaled weights, and the per-expert bucketing.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));   c_e = s_e + bias_e
//   groups of E/n_group consecutive experts: a group's score is the sum of its
//   1 or 2 largest c; experts outside the topk_group best groups are dropped
//   (ties to the lower group); the k largest c are selected in descending
//   order, ties to the lower expert; w = s at them, / their sum, * scale.
//
// Scores are kept in fp64: two experts a few 1e-8 apart, where sigmoid scores
// of a large batch meet daily, must order as their logits and biases do, not
// as fp32 rounding does.  fp64 and fp32 fma have the same rate on this chip,
// so at one exponential per expert the cost is instruction count, not width.
//
// One wave per token, lane l holding experts l, l + 64, ...: a logit row is
// read once, coalesced.  Bound: latency (one token) or the fp64 exponentials
// and k extraction rounds (a prompt chunk; the logits are 4 MB, ~1 us of HBM).
// Measured: one token of 256 experts in 8 groups 6.1 us a call, 777 tokens of
// 512 experts / top-10 14.0, 4,096 tokens of 256 experts in 8 groups 15.1.
//
// Bucketing uses that a token names an expert at most once: the tokens of a
// tile that chose e form a bit mask, so a pair's rank within its tile is a
// population count, with no serial scan over pairs.
//   * T*k <= 256: routing and bucketing in one workgroup.
//   * up to kPlaceMaxT tokens: a routing kernel per 8, 16 or 64 tokens writes
//     each tile's counts (one byte per expert) and ranks; a second kernel's
//     workgroups each sum the byte counts of all tiles (E bytes a tile, from
//     L2) and place their tiles' pairs.
//   * above that the sums every workgroup repeats would grow quadratically:
//     the tiled counting sort of route.hip (three launches) places the pairs
//     (4,096 tokens: 15.1 us with the placing kernel, 22.7 with the sort;
//     16,384: 44.2 and 53.3).
#include "fp8.h"

namespace moe {

namespace {

constexpr int kPlaceMaxT = 16384;   // 16-bit packed sums: tiles * 16 (or 64) tokens < 65536
constexpr int kRouteWaves = 16;

// DPP move of a double's halves (lanes outside row_mask, or without a source, read 0).
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint64_t lo = dpp_u<CTRL, ROW_MASK>((uint32_t)u), hi = dpp_u<CTRL, ROW_MASK>((uint32_t)(u >> 32));
    return __longlong_as_double((long long)(hi << 32 | lo));
}

// Sum over the 16 lanes of a DPP row, in each of them; over the wave, in every lane.
__device__ __forceinline__ double row16_sum_f64(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    return v + dpp_f64<0x140>(v);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v = row16_sum_f64(v);
    v += dpp_f64<0x142, 0xA>(v);
    v += dpp_f64<0x143, 0xC>(v);
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, 63), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), 63);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

// e^x for x <= 0, within a few 2^-53: x = n*ln2 + r with |r| <= ln2/2 (ln2 in two
// parts, the first of 32 bits so that n times it is exact), the
// Taylor series of e^r through r^13 (the rest is below 2^-56), times 2^n.  The
// library's exp spends its branches on arguments that do not occur here.
__device__ __forceinline__ double exp_neg(double x) {
    x = fmax(x, -800.0);   // 0 from about -745 on
    const double n = __builtin_rint(x * 1.4426950408889634074);
    double r = fma(n, -0x1.62e42feep-1, x);
    r = fma(n, -0x1.a39ef35793c76p-33, r);
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// a / b for b in [1, 2048], within a few 2^-53 (two Newton steps on the hardware reciprocal, one on the quotient).
__device__ __forceinline__ double quot_f64(double a, double b) {
    double r = __builtin_amdgcn_rcp(b);
    r = fma(fma(-b, r, 1.0), r, r);
    r = fma(fma(-b, r, 1.0), r, r);
    const double q = a * r;
    return fma(fma(-b, q, a), r, q);
}

// Larger key <=> larger value; -0 ties with +0; never 0 (0 marks an absent expert).
__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
    const uint64_t key = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
    return key ? key : 1ull;
}

// Merges the two largest (a >= b) of this lane and of its partner.
__device__ __forceinline__ void merge_top2(double& a, double& b, double oa, double ob) {
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
}

// Group scores from the E biased scores in LDS: `per` lanes (a power of two,
// per * n_group <= 64) scan one group, then merge their top one or two.
// Returns a mask with bit g * per set for every selected group g.
__device__ __forceinline__ uint64_t select_groups(const double* s_c, int E, const ScoreRule& rule, int per) {
    const int lane = threadIdx.x & (kWave - 1);
    const int S = E / rule.n_group;
    const int g = lane / per, i0 = lane - g * per;
    const double ninf = -__builtin_inf();
    double a = ninf, b = ninf;             // the two largest, a >= b
    const double* p = s_c + min(g, rule.n_group - 1) * S;
    for (int i = i0; i < S; i += 4 * per) {
        double v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = p[min(i + q * per, S - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const double x = i + q * per < S ? v[q] : ninf;
            b = fmax(b, fmin(a, x));
            a = fmax(a, x);
        }
    }
    if (per > 1) merge_top2(a, b, dpp_f64<0xB1>(a), dpp_f64<0xB1>(b));
    if (per > 2) merge_top2(a, b, dpp_f64<0x4E>(a), dpp_f64<0x4E>(b));
    if (per > 4) merge_top2(a, b, dpp_f64<0x141>(a), dpp_f64<0x141>(b));   // lanes 0-3 and 4-7 each agree by now
    if (per > 8) merge_top2(a, b, dpp_f64<0x140>(a), dpp_f64<0x140>(b));
    if (per > 16) merge_top2(a, b, __shfl_xor(a, 16, kWave), __shfl_xor(b, 16, kWave));
    const double score = rule.group_top == 2 ? a + b : a;
    const uint64_t key = order_key64(score);
    int rank = 0;
    for (int h = 0; h < rule.n_group; ++h) {
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)key, h * per);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(key >> 32), h * per);
        const uint64_t o = (uint64_t)hi << 32 | lo;
        rank += (int)(o > key) + (int)((o == key) & (h < g));
    }
    return __ballot(g < rule.n_group && i0 == 0 && rank < rule.topk_group);
}

// The k largest keys of a wave (lane l: experts l + 64*v), ties to the lower expert: lane j < k returns slot j's.
template <int V>
__device__ __forceinline__ int extract_f64(uint64_t (&key)[V], int k) {
    const int lane = threadIdx.x & (kWave - 1);
    int my_e = -1;
    for (int j = 0; j < k; ++j) {
        uint64_t best = key[0];
        int bv = 0;
#pragma unroll
        for (int v = 1; v < V; ++v) {
            const bool gt = key[v] > best;
            best = gt ? key[v] : best;
            bv = gt ? v : bv;
        }
        const uint32_t mh = wave_max_u32((uint32_t)(best >> 32));
        bool hold = (uint32_t)(best >> 32) == mh;
        const uint32_t ml = wave_max_u32(hold ? (uint32_t)best : 0u);
        hold = hold && (uint32_t)best == ml;
        const uint32_t c = ~wave_max_u32(hold ? ~(uint32_t)(kWave * bv + lane) : 0u);   // 64*v + lane is the expert
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = (uint32_t)(kWave * v + lane) == c ? 0ull : key[v];
        if (lane == j) my_e = (int)c;
    }
    return my_e;
}

// One wave selects the top-k experts of one token.  Lane j < k returns slot
// j's expert and weight (other lanes -1 and 0).  buf: E doubles of LDS that
// belong to this wave.  A NaN or infinite logit, or a bias that is NaN or
// +inf, raises kErrLogitNonFinite; the slots still hold distinct experts.
//
// The extraction is instruction-bound (a prompt chunk holds four waves a SIMD),
// and 64-bit keys double it.  Rounding to fp32 never reverses two scores, so
// the keys of the extraction are the scores in fp32 (WaveExtract, route.hip);
// only if two of the k + 1 largest round to the same fp32, about once in 10^4
// tokens, the token is extracted again by its fp64 keys.
template <int V>
__device__ __forceinline__ void wave_topk_scored(const float* __restrict__ lg, int E, int k, const ScoreRule& rule,
                                                 double* buf, int& out_e, float& out_w) {
    const int lane = threadIdx.x & (kWave - 1);
    float xv[V], bi[V];
#pragma unroll
    for (int v = 0; v < V; ++v) xv[v] = lg[min(lane + kWave * v, E - 1)];
#pragma unroll
    for (int v = 0; v < V; ++v) bi[v] = rule.bias ? rule.bias[min(lane + kWave * v, E - 1)] : 0.0f;
    double s[V];
    bool bad = false;   // the clamped duplicates of expert E - 1 say nothing new
#pragma unroll
    for (int v = 0; v < V; ++v) bad |= !isfinite(xv[v]) | !(bi[v] < __builtin_inff());
    if (rule.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) {   // e^-|l| never overflows; 1/(1 + z) or z/(1 + z)
            const double z = exp_neg(-fabs((double)xv[v]));
            s[v] = quot_f64(xv[v] >= 0.0f ? 1.0 : z, 1.0 + z);
        }
    } else {
        uint32_t mk = order_key(xv[0]);
#pragma unroll
        for (int v = 1; v < V; ++v) mk = max(mk, order_key(xv[v]));
        const double m = (double)key_value(wave_max_u32(mk));
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = exp_neg((double)xv[v] - m);
            part += lane + kWave * v < E ? s[v] : 0.0;
        }
        const double sum = wave_sum_f64(part);   // in [1, E]
        const double inv = quot_f64(1.0, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] *= inv;
    }
    if (__any(bad) && lane == 0) raise_error(kErrLogitNonFinite);

    uint64_t groups = 0;
    int lanes = 1;   // lanes that scan a group
    if (rule.n_group > 1) {
        while (2 * lanes * rule.n_group <= kWave) lanes *= 2;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + kWave * v < E) buf[lane + kWave * v] = s[v] + (double)bi[v];
        __builtin_amdgcn_wave_barrier();
        groups = select_groups(buf, E, rule, lanes);
        __builtin_amdgcn_wave_barrier();
    }
    WaveExtract<V> ex;
    uint32_t in_mask = 0;   // bit v: expert lane + 64*v takes part
    const float per = 1.0f / (float)(E / rule.n_group);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + kWave * v;
        bool in = e < E;
        // group of e: (e + 0.5)/S is at least 0.5/1024 from an integer, far above the fp32 rounding of the product
        if (rule.n_group > 1) in = in & (bool)((groups >> ((int)(((float)e + 0.5f) * per) * lanes & 63)) & 1ull);
        const uint32_t key = max(order_key((float)(s[v] + (double)bi[v])), 1u);
        ex.key[v] = in ? key : 0u;
        in_mask |= (uint32_t)in << v;
        if (e < E) buf[e] = s[v];
    }
    if constexpr (V <= kSortedV)
        ex.sort_keys();
    else
        ex.refresh();
    int my_e = -1;
    uint32_t last = 0;
    bool tie = false;
    for (int j = 0; j < k; ++j) {
        uint32_t M;
        const int e = ex.next(M);
        tie |= M == last;
        last = M;
        my_e = lane == j ? e : my_e;
    }
    if (tie || __any(ex.best == last)) {
        uint64_t key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = (in_mask >> v) & 1u ? order_key64(s[v] + (double)bi[v]) : 0ull;
        my_e = extract_f64<V>(key, k);
    }
    __builtin_amdgcn_wave_barrier();
    double w = my_e >= 0 ? buf[my_e] : 0.0;
    if (rule.renorm) {
        const double sum = row16_sum_f64(w);   // at most 16 slots: one row of lanes
        w = sum > 0.0 ? w / sum : 0.0;
    }
    out_e = my_e;
    out_w = (float)(w * (double)rule.scale);
}

// The grouped products' work list from the bucket counts and offsets (Fp8ItemList,
// fp8.h).  Every thread of the workgroup calls it (blockDim.x >= E); thread e < E
// passes expert e's, the others 0.  s_start, s_cnt, s_off: E ints of LDS each.
// A thread finds entry j's expert as the last one whose first entry is <= j
// (experts without tiles share the next one's first entry).
__device__ void write_item_list(int c, int off, int npairs, int E, const Fp8ItemList& tl, int* s_wave, int* s_start,
                                int* s_cnt, int* s_off) {
    const int tid = threadIdx.x;
    int total = 0;
    const int start = block_exclusive_scan((c + tl.mt - 1) / tl.mt, s_wave, total);
    if (tid < E) {
        s_start[tid] = start;
        s_cnt[tid] = c;
        s_off[tid] = off;
    }
    __syncthreads();
    const int ns = tl.has_shared ? (tl.T + tl.mt - 1) / tl.mt : 0;
    const int n = min(total + ns, tl.max_items);   // counts of a routing pass never exceed it
    for (int j = tid; j < n; j += blockDim.x) {
        Fp8Item it;
        if (j < total) {
            int lo = 0, hi = E - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_start[mid] <= j)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            it.e = lo;
            it.m0 = (j - s_start[lo]) * tl.mt;
            it.n_tok = min(tl.mt, s_cnt[lo] - it.m0);
            it.row0 = s_off[lo] + it.m0;
        } else {
            it.e = E;
            it.m0 = (j - total) * tl.mt;
            it.n_tok = min(tl.mt, tl.T - it.m0);
            it.row0 = npairs + it.m0;
        }
        *reinterpret_cast<int4*>(tl.items + j) = make_int4(it.e, it.m0, it.n_tok, it.row0);
    }
    if (tid == 0) {
        if (total + ns > tl.max_items) raise_error(kErrPairRange);
        *tl.n_items = n;
    }
}

// T*k <= kSmallPairs: workgroup 0 routes and buckets, the others quantise x (layer call).
template <int V, typename XT>
__global__ void __launch_bounds__(1024) route_scored_small_kernel(const float* __restrict__ logits, int T, int E, int k,
                                                                  ScoreRule rule, RoutingPtrs r, int waves, Fp8ItemList tl,
                                                                  ActQuant<XT> aq) {
    extern __shared__ double s_buf[];               // [waves][E], then mask[E][words]: a bit per token that chose e
    __shared__ __attribute__((aligned(16))) int s_idx[kSmallPairs];
    __shared__ int s_off[1024], s_cnt[1024], s_start[1024];
    __shared__ int s_wave[kWave + 1];
    if (blockIdx.x > 0) {
        aq.run(blockIdx.x - 1);
        return;
    }
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const int P = T * k;
    const bool quick = P <= kWave && tl.mt == 0;
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_buf + (int64_t)waves * E);
    const int words = (T + 31) / 32;
    if (!quick) {
        for (int i = tid; i < E * words; i += blockDim.x) s_mask[i] = 0;
        __syncthreads();
    }
    if (wave < waves) {
        for (int t = wave; t < T; t += waves) {
            int e;
            float w;
            wave_topk_scored<V>(logits + (int64_t)t * E, E, k, rule, s_buf + (int64_t)wave * E, e, w);
            if (lane < k) {
                r.idx[t * k + lane] = e;
                r.w[t * k + lane] = w;
                s_idx[t * k + lane] = e;
                if (!quick) atomicOr(&s_mask[e * words + (t >> 5)], 1u << (t & 31));
            }
        }
    }
    if (quick && tid >= P && tid < kWave) s_idx[tid] = E;   // counted by no expert
    __syncthreads();
    if (quick) {
        // few pairs: every expert counts the pairs below and at it; wave 0 places the pairs
        if (tid < E) {
            int c = 0, off = 0;
            for (int q = 0; q < P; q += 4) {
                const int4 v = *reinterpret_cast<const int4*>(s_idx + q);
                c += (v.x == tid) + (v.y == tid) + (v.z == tid) + (v.w == tid);
                off += (v.x < tid) + (v.y < tid) + (v.z < tid) + (v.w < tid);
            }
            r.count[tid] = c;
            r.offset[tid] = off;
        }
        if (wave == 0) {
            const int e = lane < P ? s_idx[lane] : E;
            int below, before, ubelow, n_uniq;
            bool first;
            wave_buckets(e, P, below, before, first, ubelow, n_uniq);
            if (lane < P) r.pair[below + before] = lane;
            if (first) r.active[ubelow] = e;
            if (lane == 0) {
                r.offset[E] = P;
                *r.n_active = n_uniq;
            }
        }
        return;
    }
    int c = 0;
    if (tid < E)
        for (int i = 0; i < words; ++i) c += __popc(s_mask[tid * words + i]);
    // one scan for both: pairs in the low half, active experts in the high half
    int total;
    const int pre = block_exclusive_scan(c | (c > 0 ? 0x10000 : 0), s_wave, total);
    if (tid < E) {
        s_off[tid] = pre & 0xFFFF;
        r.count[tid] = c;
        r.offset[tid] = pre & 0xFFFF;
        if (c > 0) r.active[pre >> 16] = tid;
    }
    if (tid == 0) {
        r.offset[E] = total & 0xFFFF;
        *r.n_active = total >> 16;
    }
    __syncthreads();
    for (int p = tid; p < P; p += blockDim.x) {
        const int e = s_idx[p], t = p / k;
        int rank = __popc(s_mask[e * words + (t >> 5)] & ((1u << (t & 31)) - 1u));
        for (int i = 0; i < (t >> 5); ++i) rank += __popc(s_mask[e * words + i]);
        r.pair[s_off[e] + rank] = p;
    }
    if (tl.mt > 0) {
        __syncthreads();   // s_off is free again
        write_item_list(c, pre & 0xFFFF, P, E, tl, s_wave, s_start, s_cnt, s_off);
    }
}

// A tile of tt tokens (8, 16 or 64): routing, the tile's byte count per expert and each pair's rank in the tile.
// Workgroups from n_route on quantise x (layer call).
template <int V, typename XT>
__global__ void __launch_bounds__(1024) route_scored_tile_kernel(const float* __restrict__ logits, int T, int E, int k,
                                                                 ScoreRule rule, int32_t* __restrict__ idx,
                                                                 float* __restrict__ w, int tt,
                                                                 uint8_t* __restrict__ hist,
                                                                 uint8_t* __restrict__ rank, int hist_ld, int n_route,
                                                                 ActQuant<XT> aq) {
    extern __shared__ double s_buf[];
    __shared__ uint32_t s_mask[1024][2];
    __shared__ int s_idx[kSmallPairs];
    if ((int)blockIdx.x >= n_route) {
        aq.run(blockIdx.x - n_route);
        return;
    }
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const int waves = blockDim.x / kWave;
    const int t0 = blockIdx.x * tt;
    for (int e = tid; e < E; e += blockDim.x) s_mask[e][0] = s_mask[e][1] = 0;
    __syncthreads();
    for (int q = wave; q < tt; q += waves) {
        const int t = t0 + q;
        if (t >= T) break;
        int e;
        float wt;
        wave_topk_scored<V>(logits + (int64_t)t * E, E, k, rule, s_buf + (int64_t)wave * E, e, wt);
        if (lane < k) {
            idx[(int64_t)t * k + lane] = e;
            w[(int64_t)t * k + lane] = wt;
            s_idx[q * k + lane] = e;
            atomicOr(&s_mask[e][q >> 5], 1u << (q & 31));
        }
    }
    __syncthreads();
    const int n = min(tt, T - t0) * k;
    for (int p = tid; p < n; p += blockDim.x) {
        const int e = s_idx[p], q = p / k;
        int rk = __popc(s_mask[e][q >> 5] & ((1u << (q & 31)) - 1u));
        if (q >= 32) rk += __popc(s_mask[e][0]);
        rank[(int64_t)t0 * k + p] = (uint8_t)rk;
    }
    for (int e = tid; e < hist_ld; e += blockDim.x)
        hist[(int64_t)blockIdx.x * hist_ld + e] = e < E ? (uint8_t)(__popc(s_mask[e][0]) + __popc(s_mask[e][1])) : 0;
}

// Workgroup b places the pairs of tiles [b*per, (b+1)*per).  Thread (g, c) sums
// dword column c (four experts' bytes) over tiles g, g + G, ... into 16-bit
// halves: before its range, and in all.  Workgroup 0 also writes count, offset and the active list.
__global__ void __launch_bounds__(1024) route_place_kernel(const int32_t* __restrict__ idx, int T, int E, int k, int tt,
                                                           int n_tiles, int per, const uint8_t* __restrict__ hist,
                                                           const uint8_t* __restrict__ rank, int hist_ld,
                                                           RoutingPtrs r, Fp8ItemList tl) {
    __shared__ uint32_t s_sum[2][1024];   // [before | all][expert]
    __shared__ int s_base[1024], s_list[1024];
    __shared__ int s_wave[kWave + 1];
    const int tid = threadIdx.x;
    const int cols = hist_ld / 4;
    const int G = blockDim.x / cols;
    const int g = tid / cols, c = tid - g * cols;
    const int first = blockIdx.x * per;
    for (int e = tid; e < 1024; e += blockDim.x) s_sum[0][e] = s_sum[1][e] = 0;
    __syncthreads();
    if (g < G) {
        uint32_t b0 = 0, b1 = 0, a0 = 0, a1 = 0;   // experts 4c + {0, 2}, {1, 3}
        const uint32_t* h = reinterpret_cast<const uint32_t*>(hist) + c;
        for (int t0 = g; t0 < n_tiles; t0 += 8 * G) {   // eight loads in flight
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = t0 + i * G < n_tiles ? h[(int64_t)(t0 + i * G) * cols] : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v0 = v[i] & 0x00FF00FFu, v1 = (v[i] >> 8) & 0x00FF00FFu;
                a0 += v0;
                a1 += v1;
                b0 += t0 + i * G < first ? v0 : 0u;
                b1 += t0 + i * G < first ? v1 : 0u;
            }
        }
        const uint32_t part[2][4] = {{b0 & 0xFFFFu, b1 & 0xFFFFu, b0 >> 16, b1 >> 16},
                                     {a0 & 0xFFFFu, a1 & 0xFFFFu, a0 >> 16, a1 >> 16}};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (part[q][i]) atomicAdd(&s_sum[q][4 * c + i], part[q][i]);   // integer: order does not matter
    }
    __syncthreads();
    const int cnt = tid < E ? (int)s_sum[1][tid] : 0;
    int total;
    const int off = block_exclusive_scan(cnt, s_wave, total);
    if (tid < E) s_base[tid] = off + (int)s_sum[0][tid];
    if (blockIdx.x == 0) {
        int n_act;
        const int apos = block_exclusive_scan(cnt > 0 ? 1 : 0, s_wave, n_act);
        if (tid < E) {
            r.count[tid] = cnt;
            r.offset[tid] = off;
            if (cnt > 0) r.active[apos] = tid;
        }
        if (tid == 0) {
            r.offset[E] = total;
            *r.n_active = n_act;
        }
        if (tl.mt > 0)
            write_item_list(cnt, off, T * k, E, tl, s_wave, reinterpret_cast<int*>(s_sum[0]),
                            reinterpret_cast<int*>(s_sum[1]), s_list);
    }
    __syncthreads();
    for (int tile = first; tile < min(first + per, n_tiles); ++tile) {
        const int64_t p0 = (int64_t)tile * tt * k;
        const int n = min(tt, T - tile * tt) * k;
        for (int p = tid; p < n; p += blockDim.x) r.pair[s_base[idx[p0 + p]] + rank[p0 + p]] = (int32_t)(p0 + p);
        __syncthreads();
        if (tid < E) s_base[tid] += hist[(int64_t)tile * hist_ld + tid];
        __syncthreads();
    }
}

// Above kPlaceMaxT tokens: routing alone, one wave per token.
template <int V>
__global__ void __launch_bounds__(256) route_scored_tokens_kernel(const float* __restrict__ logits, int T, int E, int k,
                                                                  ScoreRule rule, int32_t* __restrict__ idx,
                                                                  float* __restrict__ w) {
    extern __shared__ double s_buf[];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * (blockDim.x / kWave) + wave;
    if (t >= T) return;
    int e;
    float wt;
    wave_topk_scored<V>(logits + (int64_t)t * E, E, k, rule, s_buf + (int64_t)wave * E, e, wt);
    if (lane < k) {
        idx[(int64_t)t * k + lane] = e;
        w[(int64_t)t * k + lane] = wt;
    }
}

// The layer call's part of the routing launches: x to quantise (null: none) and the work list (mt 0: none).
template <int V, typename XT>
hipError_t route_scored_v(const float* logits, int T, int E, int k, const ScoreRule& rule, const RoutingPtrs& r,
                          void* ws, hipStream_t s, const Fp8ItemList& tl, const ActQuant<XT>& aq) {
    const int P = T * k;
    const unsigned nq = aq.x ? aq.groups() : 0;
    // one wave's score buffer is E doubles: at most 64 KB of them in a workgroup
    const int waves = E <= 512 ? kRouteWaves : kRouteWaves / 2;
    if (P <= kSmallPairs) {
        const int used = T < waves ? T : waves;
        const size_t lds = (size_t)used * E * sizeof(double) + (size_t)E * ((T + 31) / 32) * 4;
        route_scored_small_kernel<V, XT><<<1 + nq, 1024, lds, s>>>(logits, T, E, k, rule, r, used, tl, aq);
        return hipGetLastError();
    }
    if (T > kPlaceMaxT) {
        const int n_tiles = (P + kTilePairs - 1) / kTilePairs;
        int32_t* tile_hist = (int32_t*)ws;
        int32_t* rank = tile_hist + (size_t)n_tiles * E;
        route_scored_tokens_kernel<V><<<(T + 3) / 4, 256, (size_t)4 * E * sizeof(double), s>>>(logits, T, E, k, rule,
                                                                                             r.idx, r.w);
        if (aq.x) quantize_fp8_kernel<XT><<<nq, 1024, 0, s>>>(aq);
        bucket_tile_kernel<<<n_tiles, kTilePairs, 0, s>>>(r.idx, P, E, tile_hist, rank);
        bucket_scan_kernel<<<1, 1024, 0, s>>>(n_tiles, E, P, tile_hist, r, TileList{});
        bucket_scatter_kernel<<<(P + 255) / 256, 256, 0, s>>>(r.idx, P, E, tile_hist, r.offset, rank, r.pair);
        return hipGetLastError();   // the work list is left to launch_ffn_fp8
    }
    // 64-token tiles for k < 4 keep the counts within route_workspace_bytes: ceil(T/64) * E bytes there,
    // ceil(T/16) * E <= ceil(T*k/256) * E * 4 for k >= 4
    // (8-token tiles, for k >= 8, spread a batch of up to 2,048 tokens over twice the CUs: 777 tokens 11.2 us
    // against 13.4 with 16, 2,048 12.8 / 13.9, 4,096 17.8 / 15.1)
    const int tt = k < 4 ? 64 : (k >= 8 && T <= 2048 ? 8 : 16);
    const int n_tiles = (T + tt - 1) / tt;
    const int hist_ld = (E + 3) / 4 * 4;
    uint8_t* hist = (uint8_t*)ws;
    uint8_t* rank = hist + (size_t)n_tiles * hist_ld;
    // the quantising workgroups have as many threads as ActQuant::groups counts on
    const int threads = aq.x ? 1024 : (tt < waves ? tt : waves) * kWave;
    route_scored_tile_kernel<V, XT><<<n_tiles + nq, threads, (size_t)(threads / kWave) * E * sizeof(double), s>>>(
        logits, T, E, k, rule, r.idx, r.w, tt, hist, rank, hist_ld, n_tiles, aq);
    const int per = (n_tiles + 255) / 256;
    route_place_kernel<<<(n_tiles + per - 1) / per, 1024, 0, s>>>(r.idx, T, E, k, tt, n_tiles, per, hist, rank, hist_ld, r,
                                                                  tl);
    return hipGetLastError();
}

template <typename XT>
hipError_t route_scored_x(const float* logits, int T, int E, int k, const ScoreRule& rule, const RoutingPtrs& r,
                          void* ws, hipStream_t s, const Fp8ItemList& tl, const ActQuant<XT>& aq) {
    const int v = topk_vpl(E);
    if (v == 4) return route_scored_v<4, XT>(logits, T, E, k, rule, r, ws, s, tl, aq);
    if (v == 8) return route_scored_v<8, XT>(logits, T, E, k, rule, r, ws, s, tl, aq);
    return route_scored_v<16, XT>(logits, T, E, k, rule, r, ws, s, tl, aq);
}

}  // namespace

hipError_t launch_route_scored(const float* logits, int T, int E, int k, const ScoreRule& rule, const RoutingPtrs& r,
                               void* ws, hipStream_t s) {
    return route_scored_x<float>(logits, T, E, k, rule, r, ws, s, Fp8ItemList{}, ActQuant<float>{});
}

hipError_t launch_route_quantize_fp8(const float* logits, int T, int E, int k, const ScoreRule& rule,
                                     const RoutingPtrs& r, void* ws, const Fp8ItemList& tl, const void* x, ElemType xt,
                                     int H, uint8_t* xq, float* xs, hipStream_t s, bool* list_done) {
    *list_done = tl.mt > 0 && (T * k <= kSmallPairs || T <= kPlaceMaxT);
    if (xt == ElemType::kF32)
        return route_scored_x(logits, T, E, k, rule, r, ws, s, tl, ActQuant<float>(x, H, T, H, xq, xs));
    if (xt == ElemType::kF16)
        return route_scored_x(logits, T, E, k, rule, r, ws, s, tl, ActQuant<_Float16>(x, H, T, H, xq, xs));
    return route_scored_x(logits, T, E, k, rule, r, ws, s, tl, ActQuant<__bf16>(x, H, T, H, xq, xs));
}

}  // namespace moe

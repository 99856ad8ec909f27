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
//
// Bucketing uses that a token names an expert at most once: the tokens of a
// tile that chose e form a bit mask, so a pair's rank within its tile is a
// population count, with no serial scan over pairs.
//   * T*k <= 256: routing and bucketing in one workgroup.
//   * up to kPlaceMaxT tokens: a routing kernel per 16 or 64 tokens writes
//     each tile's counts (one byte per expert) and ranks; a second kernel's
//     workgroups each sum the byte counts of all tiles (E bytes a tile, from
//     L2) and place their tiles' pairs.
//   * above that the sums every workgroup repeats would grow quadratically:
//     the tiled counting sort of route.hip (three launches) places the pairs.
#include "fp8.h"

namespace moe {

namespace {

constexpr int kPlaceMaxT = 16384;   // 16-bit packed sums: tiles * 16 (or 64) tokens < 65536
constexpr int kRouteWaves = 16;

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// Larger key <=> larger value; -0 ties with +0; never 0 (0 marks an absent expert).
__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
    const uint64_t key = (u >> 63) ? ~u : (u | 0x8000000000000000ull);
    return key ? key : 1ull;
}

// Up to n_group groups' scores from the E biased scores in LDS: 64 / G lanes
// (G the next power of two >= n_group) scan one group, then merge their top
// one or two.  Returns the mask of the selected groups.
__device__ __forceinline__ uint64_t select_groups(const double* s_c, int E, const ScoreRule& rule) {
    const int lane = threadIdx.x & (kWave - 1);
    const int S = E / rule.n_group;
    int per = kWave;                       // lanes per group
    while (kWave / per < rule.n_group) per >>= 1;
    const int g = lane / per, i0 = lane - g * per;
    const double ninf = -__builtin_inf();
    double a = ninf, b = ninf;             // the two largest, a >= b
    if (g < rule.n_group) {
        for (int i = i0; i < S; i += per) {
            const double v = s_c[g * S + i];
            b = fmax(b, fmin(a, v));
            a = fmax(a, v);
        }
    }
    for (int o = 1; o < per; o <<= 1) {
        const double oa = __shfl_xor(a, o, kWave), ob = __shfl_xor(b, o, kWave);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
    }
    const double score = rule.group_top == 2 ? a + b : a;
    const uint64_t key = order_key64(score);
    int rank = 0;
    for (int h = 0; h < rule.n_group; ++h) {
        const uint64_t o = __shfl(key, h * per, kWave);
        rank += (o > key) || (o == key && h < g);
    }
    const bool sel = g < rule.n_group && i0 == 0 && rank < rule.topk_group;
    const uint64_t lanes = __ballot(sel);
    uint64_t mask = 0;
    for (int h = 0; h < rule.n_group; ++h) mask |= ((lanes >> (h * per)) & 1ull) << h;
    return mask;
}

// One wave selects the top-k experts of one token.  Lane j < k returns slot
// j's expert and weight (other lanes -1 and 0).  buf: E doubles of LDS that
// belong to this wave.  A NaN or infinite logit, or a bias that is NaN or
// +inf, raises kErrLogitNonFinite; the slots still hold distinct experts.
template <int V>
__device__ __forceinline__ void wave_topk_scored(const float* __restrict__ lg, int E, int k, const ScoreRule& rule,
                                                 double* buf, int& out_e, float& out_w) {
    const int lane = threadIdx.x & (kWave - 1);
    float xv[V], bi[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = min(lane + kWave * v, E - 1);
        xv[v] = lg[e];
        bi[v] = rule.bias ? rule.bias[e] : 0.0f;
    }
    double s[V];
    bool bad = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool in = lane + kWave * v < E;
        bad |= in & (!isfinite(xv[v]) | !(bi[v] < __builtin_inff()));
    }
    if (rule.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 1.0 / (1.0 + exp(-(double)xv[v]));
    } else {
        float m = xv[0];   // the clamped duplicates of expert E - 1 do not move a maximum
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, xv[v]);
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = lane + kWave * v < E ? exp((double)xv[v] - (double)m) : 0.0;
            part += s[v];
        }
        const double inv = 1.0 / wave_sum_f64(part);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] *= inv;
    }
    if (__any(bad) && lane == 0) raise_error(kErrLogitNonFinite);

    uint64_t groups = ~0ull;
    if (rule.n_group > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + kWave * v < E) buf[lane + kWave * v] = s[v] + (double)bi[v];
        __builtin_amdgcn_wave_barrier();
        groups = select_groups(buf, E, rule);
        __builtin_amdgcn_wave_barrier();
    }
    const int S = E / rule.n_group;
    uint64_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + kWave * v;
        const bool in = e < E && (rule.n_group == 1 || ((groups >> (e / S)) & 1ull));
        key[v] = in ? order_key64(s[v] + (double)bi[v]) : 0ull;
        if (e < E) buf[e] = s[v];
    }
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
        // wave maximum of the upper words; the lower words and the index only decide among its holders
        const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
        const uint32_t mh = wave_max_u32(hi);
        bool hold = hi == mh;
        uint64_t lanes = __ballot(hold);
        if (__popcll(lanes) != 1) {
            const uint32_t ml = wave_max_u32(hold ? lo : 0u);
            hold = hold && lo == ml;
            const uint32_t c = ~wave_max_u32(hold ? ~(uint32_t)(kWave * bv + lane) : 0u);
            lanes = 1ull << (c & (kWave - 1));
        }
        const int wl = (int)__builtin_ctzll(lanes);
        const int wv = __builtin_amdgcn_readlane(bv, wl);
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = (lane == wl && v == wv) ? 0ull : key[v];
        if (lane == j) my_e = wl + kWave * wv;
    }
    __builtin_amdgcn_wave_barrier();
    double w = my_e >= 0 ? buf[my_e] : 0.0;
    if (rule.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    out_e = my_e;
    out_w = (float)(w * (double)rule.scale);
}

// T*k <= kSmallPairs: one workgroup.  mask[e] holds one bit per token that chose e.
template <int V>
__global__ void __launch_bounds__(1024) route_scored_small_kernel(const float* __restrict__ logits, int T, int E, int k,
                                                                  ScoreRule rule, RoutingPtrs r, int waves) {
    extern __shared__ double s_buf[];               // [waves][E]
    __shared__ uint32_t s_mask[8 * 1024];           // [E][words]
    __shared__ int s_idx[kSmallPairs];
    __shared__ int s_off[1024];
    __shared__ int s_wave[kWave + 1];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid & (kWave - 1);
    const int words = (T + 31) / 32;
    for (int i = tid; i < E * words; i += blockDim.x) s_mask[i] = 0;
    __syncthreads();
    if (wave < waves) {
        for (int t = wave; t < T; t += waves) {
            int e;
            float w;
            wave_topk_scored<V>(logits + (int64_t)t * E, E, k, rule, s_buf + (int64_t)wave * E, e, w);
            if (lane < k) {
                r.idx[t * k + lane] = e;
                r.w[t * k + lane] = w;
                s_idx[t * k + lane] = e;
                atomicOr(&s_mask[e * words + (t >> 5)], 1u << (t & 31));
            }
        }
    }
    __syncthreads();
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
    for (int p = tid; p < T * k; p += blockDim.x) {
        const int e = s_idx[p], t = p / k;
        int rank = __popc(s_mask[e * words + (t >> 5)] & ((1u << (t & 31)) - 1u));
        for (int i = 0; i < (t >> 5); ++i) rank += __popc(s_mask[e * words + i]);
        r.pair[s_off[e] + rank] = p;
    }
}

// A tile of tt tokens (16 or 64): routing, the tile's byte count per expert and each pair's rank in the tile.
template <int V>
__global__ void __launch_bounds__(1024) route_scored_tile_kernel(const float* __restrict__ logits, int T, int E, int k,
                                                                 ScoreRule rule, int32_t* __restrict__ idx,
                                                                 float* __restrict__ w, int tt,
                                                                 uint8_t* __restrict__ hist,
                                                                 uint8_t* __restrict__ rank, int hist_ld) {
    extern __shared__ double s_buf[];
    __shared__ uint32_t s_mask[1024][2];
    __shared__ int s_idx[kSmallPairs];
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
                                                           RoutingPtrs r) {
    __shared__ uint32_t s_sum[2][1024];   // [before | all][expert]
    __shared__ int s_base[1024];
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
        int t = g;
        for (; t < n_tiles; t += G) {
            const uint32_t v = h[(int64_t)t * cols];
            const uint32_t v0 = v & 0x00FF00FFu, v1 = (v >> 8) & 0x00FF00FFu;
            a0 += v0;
            a1 += v1;
            b0 += t < first ? v0 : 0u;
            b1 += t < first ? v1 : 0u;
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

template <int V>
hipError_t route_scored_v(const float* logits, int T, int E, int k, const ScoreRule& rule, const RoutingPtrs& r,
                          void* ws, hipStream_t s) {
    const int P = T * k;
    // one wave's score buffer is E doubles: at most 64 KB of them in a workgroup
    const int waves = E <= 512 ? kRouteWaves : kRouteWaves / 2;
    if (P <= kSmallPairs) {
        const int used = T < waves ? T : waves;
        route_scored_small_kernel<V><<<1, 1024, (size_t)used * E * sizeof(double), s>>>(logits, T, E, k, rule, r, used);
        return hipGetLastError();
    }
    if (T > kPlaceMaxT) {
        const int n_tiles = (P + kTilePairs - 1) / kTilePairs;
        int32_t* tile_hist = (int32_t*)ws;
        int32_t* rank = tile_hist + (size_t)n_tiles * E;
        route_scored_tokens_kernel<V><<<(T + 3) / 4, 256, (size_t)4 * E * sizeof(double), s>>>(logits, T, E, k, rule,
                                                                                             r.idx, r.w);
        bucket_tile_kernel<<<n_tiles, kTilePairs, 0, s>>>(r.idx, P, E, tile_hist, rank);
        bucket_scan_kernel<<<1, 1024, 0, s>>>(n_tiles, E, P, tile_hist, r, TileList{});
        bucket_scatter_kernel<<<(P + 255) / 256, 256, 0, s>>>(r.idx, P, E, tile_hist, r.offset, rank, r.pair);
        return hipGetLastError();
    }
    // 64-token tiles for k < 4 keep the counts within route_workspace_bytes: ceil(T/64) * E bytes there,
    // ceil(T/16) * E <= ceil(T*k/256) * E * 4 for k >= 4
    const int tt = k < 4 ? 64 : 16;
    const int n_tiles = (T + tt - 1) / tt;
    const int hist_ld = (E + 3) / 4 * 4;
    uint8_t* hist = (uint8_t*)ws;
    uint8_t* rank = hist + (size_t)n_tiles * hist_ld;
    route_scored_tile_kernel<V><<<n_tiles, waves * kWave, (size_t)waves * E * sizeof(double), s>>>(
        logits, T, E, k, rule, r.idx, r.w, tt, hist, rank, hist_ld);
    const int per = (n_tiles + 255) / 256;
    route_place_kernel<<<(n_tiles + per - 1) / per, 1024, 0, s>>>(r.idx, T, E, k, tt, n_tiles, per, hist, rank, hist_ld, r);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const float* logits, int T, int E, int k, const ScoreRule& rule, const RoutingPtrs& r,
                               void* ws, hipStream_t s) {
    const int v = topk_vpl(E);
    if (v == 4) return route_scored_v<4>(logits, T, E, k, rule, r, ws, s);
    if (v == 8) return route_scored_v<8>(logits, T, E, k, rule, r, ws, s);
    return route_scored_v<16>(logits, T, E, k, rule, r, ws, s);
}

}  // namespace moe

// logprobs.hip -- log probabilities of given tokens, entropy and the most
// probable tokens of rows of logits, in one pass over them.
//
// Each lane keeps a running maximum m, the sum s of e = 2^y with y = (x - m)
// log2(e), and the sum t of e y, which is what the entropy needs:
// H = ln s - ln 2 * t / s.
// One step a logit gives y' = x log2(e) + F32's -m log2(e), which is rounded by up to
// half a unit in its last place: by little at ordinary logits, by 0.06 at a million,
// by more than F32's exponents at masks of -1e10.  y - y' is the same for all x, and
// one FMA has it exactly (`low`): it counts where sums move to another maximum, and
// at the end they are brought to y.  Where it could pass 1, from 2^24 on, the maximum
// is subtracted first, at two steps a logit.
// The most probable tokens cost the pass nothing: its 256 lanes' maxima are there
// at its end, and what the n-th largest of them is, at least n elements reach.
// A lane keeps a maximum for each of its four loads of a piece as well: those that
// reach the bound (n, and few more) have their elements looked through again, about
// n / 1024 of the row, though in whole lines of 128 bytes n / 128; the elements that
// reach it, little more than n, go to LDS as 64-bit keys (value, then the lower
// token), where each counts the larger ones: its place.  Where more reach it than there is room for (many equal
// logits), all elements go through a list in a register, one lane a place.
// Rows are a workgroup's each; those of a last round that would leave much of the
// chip empty are split, and a second launch joins their parts.
//
// Bound by HBM when large: 2048 rows of 152064 in BF16, the 8 best, take 122 us, 5.1
// TB/s (5 us more where the maxima are a lane's alone, and its four loads of a piece
// are looked through: a fifth more bytes; 2 less without what `low` costs).  Small
// calls are two launches and their trips to memory: 12 us for one such row, 11 for 16
// rows of 129281 in F32.
#include "qp_device.hpp"
#include "qp_launch.hpp"
#include "decoder.hpp"

namespace qp {
namespace {

constexpr uint32_t WAVES = 4, WG = 64 * WAVES;
constexpr int NV = 4;                      // 16-byte loads of a lane and piece
constexpr uint32_t RESIDENT = 8;           // workgroups that a compute unit holds at a time
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// A part's results: sums, and (behind all parts' sums) the list of `top` keys.
struct Sums {
    float m, s, t, pad;
};

// Larger key: larger value, or the same and a lower token; never 0.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);       // -0 as +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u)
{
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}

// The wave's list: lane i holds the i-th largest key (0: none yet).
struct List {
    uint64_t key;
    __device__ __forceinline__ void insert(uint64_t k, uint32_t lane)
    {
        const uint32_t place = __popcll(__ballot(key > k));
        constexpr int SHR = 0x138;                      // from the lane below
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)key, SHR, 0xf, 0xf, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(key >> 32), SHR, 0xf, 0xf, false);
        key = lane < place ? key : lane == place ? k : (uint64_t)hi << 32 | lo;
    }
    __device__ __forceinline__ uint64_t at(uint32_t i) const
    {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i) << 32 |
               (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, i);
    }
};

// Enters what passes the `top`-th of the list, `least`, from a key a lane.
__device__ __forceinline__ void merge(List &best, uint64_t &least, uint64_t k, uint32_t top, uint32_t lane)
{
    for (uint64_t who = __ballot(k > least); who; who &= who - 1) {
        const uint64_t c = List{k}.at(__builtin_ctzll(who));
        if (c > least) {
            best.insert(c, lane);
            least = best.at(top - 1);
        }
    }
}

// Room in LDS for keys that reach a bound, and for the largest in order.
constexpr uint32_t ROOM = 512;
constexpr uint32_t BATCH = 16;
struct Bench {
    uint64_t in[ROOM + BATCH], out[64];
    uint32_t n;                            // keys that reached it: more than ROOM are not all there
    uint32_t loads;                        // entries of the list of loads to look through
};

__device__ __forceinline__ void collect(Bench &bench, uint64_t key)
{
    const uint32_t at = atomicAdd(&bench.n, 1u);        // (in any order: they are put in order by value)
    if (at < ROOM)
        bench.in[at] = key;
}

// The `top` largest of the n <= ROOM collected keys to bench.out, by `threads`
// threads (at least BATCH): each key counts the larger ones, BATCH at a time.
__device__ __forceinline__ void in_order(Bench &bench, uint32_t n, uint32_t top, uint32_t thread, uint32_t threads)
{
    if (thread < BATCH)
        bench.in[n + thread] = 0;          // no key
    if (threads == 64)
        __builtin_amdgcn_wave_barrier();
    else
        __syncthreads();
    for (uint32_t i0 = thread; i0 < n; i0 += threads) {
        const uint64_t mine = bench.in[i0];
        uint32_t place = 0;
        for (uint32_t i = 0; i < n; i += BATCH) {
            uint64_t k[BATCH];
#pragma unroll
            for (uint32_t j = 0; j < BATCH; ++j)
                k[j] = bench.in[i + j];
#pragma unroll
            for (uint32_t j = 0; j < BATCH; ++j)
                place += k[j] > mine;
        }
        if (place < top)
            bench.out[place] = mine;
    }
}

// -m log2(e) less F32's of it, exactly.
__device__ __forceinline__ float low(float m) { return __builtin_fmaf(-m, LOG2E, m * LOG2E); }

// The sums s and t of y's that all grow by `by` (to another maximum, mostly far
// down: what then is nothing in F32 is 0 in both).
__device__ __forceinline__ void fade(float by, float &s, float &t)
{
    if (s > 0.0f) {
        const float f = __builtin_amdgcn_exp2f(by);
        t = f > 0.0f ? f * __builtin_fmaf(by, s, t) : 0.0f;
        s *= f;
    }
}
__device__ __forceinline__ void fade_to(float to, float m, float &s, float &t) { fade((m - to) * LOG2E, s, t); }

__device__ __forceinline__ float sum_over_wave(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off, WAVE);
    return v;
}

// One wave: the list of `parts` lists of `top` keys each, in order.  With
// h = ceil(top / lists), a value that the h-th keys of ceil(top / h) lists reach is
// reached by `top` keys: the largest such is the bound.
__device__ __forceinline__ List join_lists(const uint64_t *keys, uint32_t parts, uint32_t top, Bench &bench, uint32_t lane)
{
    const uint32_t lists = min(parts, 64u), h = (top + lists - 1) / lists, need = (top + h - 1) / h, total = parts * top;
    constexpr int U = 8;                   // loads on their way together
    uint64_t k[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        k[u] = 64 * u + lane < total ? keys[64 * u + lane] : 0;
    const uint32_t value = lane < lists ? (uint32_t)(keys[lane * top + h - 1] >> 32) : 0;
    bench.n = 0;
    bench.out[lane] = 0;
    uint32_t bits = 0;
    for (uint32_t bit = 1u << 31; bit; bit >>= 1)
        if ((uint32_t)__popcll(__ballot(value >= (bits | bit))) >= need)
            bits |= bit;
    const uint64_t bound = (uint64_t)bits << 32;
    __builtin_amdgcn_wave_barrier();
    for (uint32_t i0 = 0; i0 < total; i0 += 64 * U) {
        if (i0 != 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                k[u] = i0 + 64 * u + lane < total ? keys[i0 + 64 * u + lane] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k[u] != 0 && k[u] >= bound)
                collect(bench, k[u]);
    }
    __builtin_amdgcn_wave_barrier();
    const uint32_t n = __builtin_amdgcn_readfirstlane(bench.n);
    if (n <= ROOM) {
        in_order(bench, n, top, lane, 64);
        __builtin_amdgcn_wave_barrier();
        return {bench.out[lane]};
    }
    // more than there is room for (many equal logits): one after the other
    List best = {lane < top ? keys[lane] : 0};
    uint64_t least = best.at(top - 1);
    for (uint32_t i = top; i < parts * top; i += 64)
        merge(best, least, i + lane < parts * top ? keys[i + lane] : 0, top, lane);
    return best;
}

// A row's target: whether it is a token, and its logit.
struct Target {
    bool there;
    float x;
};
template <bool F32>
__device__ __forceinline__ Target target_of(const LogprobArgs &a, uint32_t row)
{
    Target r = {false, 0.0f};
    if (a.targets) {
        const uint32_t id = (uint32_t)a.targets[row];
        r.there = id < a.vocab;
        const size_t e = (size_t)row * a.vocab + (r.there ? id : 0);
        r.x = F32 ? ((const float *)a.logits)[e] : __uint_as_float((uint32_t)((const uint16_t *)a.logits)[e] << 16);
    }
    return r;
}

// One wave: joins `parts` sums and writes the row's outputs.
template <bool F32>
__device__ __forceinline__ void finish(const LogprobArgs &a, uint32_t row, const Sums *sums, uint32_t parts, List best,
                                       Target given, uint32_t lane)
{
    float m = -INFINITY, s = 0.0f, t = 0.0f;
    for (uint32_t i = lane; i < parts; i += 64) {
        Sums p = sums[i];
        const float to = __builtin_fmaxf(m, p.m);
        fade_to(to, m, s, t);
        fade_to(to, p.m, p.s, p.t);
        m = to;
        s += p.s;
        t += p.t;
    }
    const float top = wave_max(m);
    fade_to(top, m, s, t);
    s = sum_over_wave(s);
    t = sum_over_wave(t);
    const float base = top == -INFINITY ? 0.0f : top;
    const float norm = s == 0.0f ? 0.0f : logf(s);
    if (lane == 0) {
        if (a.targets)
            a.logprob[row] = given.there ? given.x - base - norm : 0.0f;
        if (a.entropy)
            a.entropy[row] = s == 0.0f ? 0.0f : norm - LN2 * (t / s);
    }
    if (a.top == 0)
        return;
    if (lane < a.top) {
        const uint32_t id = 0xFFFFFFFFu - (uint32_t)best.key;
        // a row with NaN may have fewer than `top` values that compare
        a.ids[(size_t)row * a.top + lane] = id < a.vocab ? (int32_t)id : 0;
        a.top_logprobs[(size_t)row * a.top + lane] =
            id < a.vocab ? from_ordered((uint32_t)(best.key >> 32)) - base - norm : __builtin_nanf("");
    }
}

// 16 bytes of logits as values; the elements at and behind `end` and before
// `begin` (they are not read) as -inf.
template <bool F32>
__device__ __forceinline__ u32x4 load16(const void *logits, uint32_t at, uint32_t begin, uint32_t end)
{
    constexpr uint32_t V = F32 ? 4 : 8;
    if (at >= begin && at + V <= end)
        return *(const u32x4 *)((const uint8_t *)logits + (size_t)at * (F32 ? 4 : 2));
    u32x4 raw;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F32) {
            raw[j] = at + j >= begin && at + j < end ? ((const uint32_t *)logits)[at + j] : 0xFF800000u;
        } else {
            const uint32_t g = at + 2 * j;
            const uint32_t lo = g >= begin && g < end ? ((const uint16_t *)logits)[g] : 0xFF80u;
            const uint32_t hi = g + 1 >= begin && g + 1 < end ? ((const uint16_t *)logits)[g + 1] : 0xFF80u;
            raw[j] = hi << 16 | lo;
        }
    }
    return raw;
}
template <bool F32>
__device__ __forceinline__ void values(u32x4 raw, float *x)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F32) {
            x[j] = __uint_as_float(raw[j]);
        } else {
            x[2 * j] = bf16_lo(raw[j]);
            x[2 * j + 1] = bf16_hi(raw[j]);
        }
    }
}

// What a workgroup has of a row: pieces of 64 x NV x 16 bytes, wave w's at
// first + PIECE * w and every `stride` from there.
template <bool F32>
struct Part {
    static constexpr uint32_t V = F32 ? 4 : 8;          // elements of 16 bytes
    static constexpr uint32_t PIECE = 64 * NV * V;
    uint32_t begin, end;                                // the row, below 2^31
    uint32_t first, stride;
};

// The whole workgroup: the `top` largest elements of its part, in order, to
// bench.out (0 behind them, where there are fewer).  m: the lane's maxima, by load.
template <bool F32>
__device__ __forceinline__ void largest(const LogprobArgs &a, const Part<F32> &p, const float *m, float *lane_max,
                                        uint16_t *loads, uint64_t *keys, Bench &bench, uint32_t lane, uint32_t wave)
{
    constexpr uint32_t V = Part<F32>::V, PIECE = Part<F32>::PIECE;
    const uint32_t tid = threadIdx.x;
    static_assert(NV == 4, "the maximum of four");
    lane_max[tid] = __builtin_fmaxf(__builtin_fmaxf(m[0], m[1]), __builtin_fmaxf(m[2], m[3]));
    if (tid < 64)
        bench.out[tid] = 0;
    if (tid == 0)
        bench.n = bench.loads = 0;
    __syncthreads();
    // the largest value with 16 zeros behind it that `top` lanes' maxima reach
    uint32_t u[WAVES], bound = 0;
#pragma unroll
    for (uint32_t w = 0; w < WAVES; ++w)
        u[w] = ordered(lane_max[64 * w + lane]);
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
        uint32_t n = 0;
#pragma unroll
        for (uint32_t w = 0; w < WAVES; ++w)
            n += __popcll(__ballot(u[w] >= (bound | bit)));
        if (n >= a.top)
            bound |= bit;
    }
    // below -inf lie the keys that are no numbers.  With -inf the elements that are
    // more are looked for, and then the first tokens that are not
    const bool rest = bound <= ordered(-INFINITY);
    const uint32_t reach = rest ? ordered(-INFINITY) + 1 : bound;
    // the loads that reach it (in any order: the elements are put in theirs)
    uint64_t who[NV];
    uint32_t mine = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        who[v] = __ballot(ordered(m[v]) >= reach);
        mine += __popcll(who[v]);
    }
    uint32_t to = 0;
    if (lane == 0 && mine != 0)
        to = atomicAdd(&bench.loads, mine);
    to = __builtin_amdgcn_readfirstlane(to);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (who[v] >> lane & 1)
            loads[to + __popcll(who[v] & ((1ull << lane) - 1))] = (uint16_t)(tid * NV + v);
        to += __popcll(who[v]);
    }
    __syncthreads();
    const uint32_t some = bench.loads;
    const uint32_t pieces = (p.end - p.first + p.stride - 1) / p.stride;    // of the first wave; p.first < p.end
    for (uint32_t i = tid; i < some * pieces; i += WG) {
        const uint32_t t = loads[i % some] / NV, v = loads[i % some] % NV;
        const uint32_t at = p.first + PIECE * (t / 64) + i / some * p.stride + (64 * v + t % 64) * V;
        if (at >= p.end)
            continue;
        float x[V];
        values<F32>(load16<F32>(a.logits, at, p.begin, p.end), x);
#pragma unroll
        for (uint32_t j = 0; j < V; ++j)
            if (ordered(x[j]) >= reach && x[j] == x[j])
                collect(bench, (uint64_t)ordered(x[j]) << 32 | (0xFFFFFFFFu - (at + j - p.begin)));
    }
    __syncthreads();
    uint32_t n = bench.n;
    bool all = n <= ROOM;
    if (rest && all) {
        // of the part's first top + n tokens, `top` are -inf
        const uint32_t from = max(p.first, p.begin);
        all = a.top + n <= PIECE - V;
        __syncthreads();
        for (uint32_t i = from + tid; all && i < min(from + a.top + n, p.end); i += WG) {
            const float x = F32 ? ((const float *)a.logits)[i]
                                : __uint_as_float((uint32_t)((const uint16_t *)a.logits)[i] << 16);
            if (x == -INFINITY)
                collect(bench, (uint64_t)ordered(x) << 32 | (0xFFFFFFFFu - (i - p.begin)));
        }
        __syncthreads();
        n = bench.n;
        all = all && n <= ROOM;
    }
    if (all) {
        in_order(bench, n, a.top, tid, WG);
        __syncthreads();
        return;
    }
    // one after the other, a list a wave
    List best = {0};
    uint64_t least = 0;
#pragma unroll 1
    for (uint32_t at = p.first + PIECE * wave; at < p.end; at += p.stride)
#pragma unroll 1
        for (int v = 0; v < NV; ++v) {
            const uint32_t f = at + (64 * v + lane) * V;
            float x[V];
            values<F32>(load16<F32>(a.logits, f, p.begin, p.end), x);
#pragma unroll
            for (uint32_t j = 0; j < V; ++j) {
                const bool in = f + j >= p.begin && f + j < p.end && x[j] == x[j];
                merge(best, least, in ? (uint64_t)ordered(x[j]) << 32 | (0xFFFFFFFFu - (f + j - p.begin)) : 0, a.top, lane);
            }
        }
    if (lane < a.top)
        keys[wave * a.top + lane] = best.key;
    __syncthreads();
    if (wave == 0) {
        best = join_lists(keys, WAVES, a.top, bench, lane);
        bench.out[lane] = lane < a.top ? best.key : 0;
    }
    __syncthreads();
}

// The first `whole` rows are a workgroup's each, the others `split` workgroups'.
// WITH_T: the entropy's sum is kept.
template <bool F32, bool WITH_T>
__global__ __launch_bounds__(WG, RESIDENT) void k_logprobs(LogprobArgs a, uint32_t whole, uint32_t split)
{
    constexpr uint32_t V = Part<F32>::V, PIECE = Part<F32>::PIECE;
    __shared__ Sums sums[WAVES];
    __shared__ float lane_max[WG];
    __shared__ uint16_t loads[WG * NV];
    __shared__ uint64_t keys[WAVES * 32];
    __shared__ Bench bench;
    const bool alone = blockIdx.x < whole;
    const uint32_t parts = alone ? 1 : split, nth = blockIdx.x - whole;
    const uint32_t row = alone ? blockIdx.x : whole + nth / split, part = alone ? 0 : nth % split;
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    Part<F32> p;
    p.begin = row * a.vocab;
    p.end = p.begin + a.vocab;
    p.first = p.begin / V * V + PIECE * WAVES * part;
    p.stride = PIECE * WAVES * parts;

    u32x4 raw[NV];
    auto load = [&](uint32_t at) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            raw[v] = load16<F32>(a.logits, at + (64 * v + lane) * V, p.begin, p.end);
    };
    Target given = {false, 0.0f};
    if (parts == 1 && wave == 0)
        given = target_of<F32>(a, row);
    float m = -INFINITY, s = 0.0f, t = 0.0f, most_of[NV];
    bool quick = false;                    // the sums are those of y' (in all lanes)
#pragma unroll
    for (int v = 0; v < NV; ++v)
        most_of[v] = -INFINITY;
    uint32_t pos = p.first + PIECE * wave;
    if (pos < p.end)
        load(pos);
    for (; pos < p.end; pos += p.stride) {
        float x[NV][V], top = -INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            values<F32>(raw[v], x[v]);
#pragma unroll
            for (uint32_t j = 0; j < V; ++j)
                most_of[v] = __builtin_fmaxf(most_of[v], x[v][j]);
            top = __builtin_fmaxf(top, most_of[v]);
        }
        if (pos + p.stride < p.end)
            load(pos + p.stride);
        const float to = __builtin_fmaxf(m, top);
        // -200 stands for all that is nothing in F32, so that -inf adds 0 and not NaN to t
        if (__all(__builtin_fabsf(to) < 0x1p24f)) {
            const float by = -to * LOG2E;
            fade(__builtin_fmaf(m - to, LOG2E, (quick ? low(m) : 0.0f) - low(to)), s, t);
            quick = true;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (uint32_t j = 0; j < V; ++j) {
                    const float y = WITH_T ? __builtin_fmaxf(__builtin_fmaf(x[v][j], LOG2E, by), -200.0f)
                                           : __builtin_fmaf(x[v][j], LOG2E, by);
                    const float e = __builtin_amdgcn_exp2f(y);
                    s += e;
                    if (WITH_T)
                        t = __builtin_fmaf(e, y, t);
                }
        } else {
            fade(__builtin_fmaf(m - to, LOG2E, quick ? low(m) : 0.0f), s, t);
            quick = false;
            const float by = to == -INFINITY ? 0.0f : to;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (uint32_t j = 0; j < V; ++j) {
                    const float y = __builtin_fmaxf((x[v][j] - by) * LOG2E, -200.0f);
                    const float e = __builtin_amdgcn_exp2f(y);
                    s += e;
                    t = __builtin_fmaf(e, y, t);
                }
        }
        m = to;
    }
    if (quick)
        fade(low(m), s, t);

    const float most = wave_max(m);
    if (a.top != 0)
        largest<F32>(a, p, most_of, lane_max, loads, keys, bench, lane, wave);
    fade_to(most, m, s, t);
    s = sum_over_wave(s);
    t = sum_over_wave(t);
    if (lane == 0)
        sums[wave] = {most, s, t, 0.0f};
    __syncthreads();
    if (wave != 0)
        return;
    const List best = {a.top != 0 ? bench.out[lane] : 0};
    if (parts == 1) {
        finish<F32>(a, row, sums, WAVES, best, given, lane);
        return;
    }
    // the workgroup's sums and list, for the join
    float top = most;
    for (uint32_t u = 1; u < WAVES; ++u)
        top = __builtin_fmaxf(top, sums[u].m);
    fade_to(top, most, s, t);
    for (uint32_t u = 1; u < WAVES; ++u) {
        Sums q = sums[u];
        fade_to(top, q.m, q.s, q.t);
        s += q.s;
        t += q.t;
    }
    Sums *to_sums = (Sums *)a.work;
    uint64_t *to_keys = (uint64_t *)(to_sums + (size_t)(gridDim.x - whole));
    if (lane == 0)
        to_sums[nth] = {top, s, t, 0.0f};
    if (lane < a.top)
        to_keys[(size_t)nth * a.top + lane] = best.key;
}

template <bool F32>
__global__ __launch_bounds__(64) void k_logprobs_join(LogprobArgs a, uint32_t parts)
{
    __shared__ Bench bench;
    const Sums *sums = (const Sums *)a.work;
    const uint64_t *keys = (const uint64_t *)(sums + (size_t)gridDim.x * parts);
    const size_t first = (size_t)blockIdx.x * parts;
    const uint32_t row = a.rows - gridDim.x + blockIdx.x;
    const Target given = target_of<F32>(a, row);
    List best = {0};
    if (a.top != 0)
        best = join_lists(keys + first * a.top, parts, a.top, bench, threadIdx.x);
    finish<F32>(a, row, sums + first, parts, best, given, threadIdx.x);
}

// How rows are dealt: a workgroup each, as long as they fill the chip; the rows of
// a last round that would leave much of it empty are split, at most until each wave
// has one piece.
struct Deal {
    uint32_t whole, split;                 // rows that are not split; parts of the others
    uint64_t parts(uint32_t rows) const { return (uint64_t)(rows - whole) * split; }
};
Deal deal(uint32_t rows, uint32_t vocab, bool f32)
{
    const uint32_t room = RESIDENT * (cu_count() ? cu_count() : 256), piece = 64 * NV * (f32 ? 4 : 8) * WAVES;
    const uint32_t last = rows % room, split = last ? min((vocab + piece - 1) / piece, room / last) : 1;
    return split > 1 ? Deal{rows - last, split} : Deal{rows, 1};
}

template <bool F32>
void launch(const LogprobArgs &a, hipStream_t st)
{
    const Deal d = deal(a.rows, a.vocab, F32);
    const dim3 grid(d.whole + (uint32_t)d.parts(a.rows));
    if (a.entropy)
        k_logprobs<F32, true><<<grid, WG, 0, st>>>(a, d.whole, d.split);
    else
        k_logprobs<F32, false><<<grid, WG, 0, st>>>(a, d.whole, d.split);
    count_launch();
    if (d.whole < a.rows) {
        k_logprobs_join<F32><<<a.rows - d.whole, 64, 0, st>>>(a, d.split);
        count_launch();
    }
}

} // namespace

uint64_t token_logprobs_work(uint32_t rows, uint32_t vocab, uint32_t top)
{
    const uint64_t parts = max(deal(rows, vocab, false).parts(rows), deal(rows, vocab, true).parts(rows));
    return max(parts * (sizeof(Sums) + 8 * top), (uint64_t)16);
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t st)
{
    if (a.f32)
        launch<true>(a, st);
    else
        launch<false>(a, st);
    return hipGetLastError();
}

} // namespace qp

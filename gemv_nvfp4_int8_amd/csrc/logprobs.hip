// logprobs.hip -- log probabilities of given tokens, entropy and the most
// probable tokens of rows of logits, in one pass over them.
//
// A wave goes through its pieces of a row 64 x NV x 16 bytes at a time and needs
// nobody else until its end.  Each lane keeps a running maximum m, the sum s of
// e = 2^y with y = (x - m) log2(e), and the sum t of e y, which is what the
// entropy needs: H = ln s - ln 2 * t / s.  The largest logits of the wave so far
// lie in a register, the i-th in lane i, as 64-bit keys (value, then the lower
// token).  The first piece's are found by a bound that as many lanes' maxima
// reach as are wanted (halving over the bits of the maxima), the few elements
// that reach it being put into LDS, where each counts the larger ones: its place.
// From then on an element enters only if it passes the last of the list, a ballot
// counts its place and the rest moves up one lane.  The four waves of a workgroup
// join through LDS, where again all keys that pass a bound count the larger ones;
// where a row a workgroup would fill the chip badly, rows are split, and a second
// launch joins the parts.
#include "qp_device.hpp"
#include "qp_launch.hpp"
#include "decoder.hpp"

namespace qp {
namespace {

constexpr uint32_t WAVES = 4, WG = 64 * WAVES;
constexpr int NV = 4;                      // 16-byte loads of a lane and piece
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

// A wave's room in LDS for keys that pass a bound, and for them in order.
constexpr uint32_t ROOM = 256;
struct Bench {
    uint64_t in[ROOM], out[64];
};

// Puts the lanes' keys that reach `bound` behind the first n; returns the new n,
// which may be more than there is room for (then not all are there).
__device__ __forceinline__ uint32_t collect(Bench &bench, uint32_t n, bool pass, uint64_t key)
{
    const uint64_t who = __ballot(pass);
    const uint32_t at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (pass && at < ROOM)
        bench.in[at] = key;
    return n + __popcll(who);
}

// The list of n <= ROOM collected keys: each counts the larger ones.
__device__ __forceinline__ List in_order(Bench &bench, uint32_t n, uint32_t lane)
{
    __builtin_amdgcn_wave_barrier();
    for (uint32_t i0 = 0; i0 < n; i0 += 64) {
        const uint64_t mine = i0 + lane < n ? bench.in[i0 + lane] : 0;
        uint32_t place = 0;
#pragma unroll 4
        for (uint32_t i = 0; i < n; ++i)
            place += bench.in[i] > mine;
        if (mine && place < 64)
            bench.out[place] = mine;
    }
    __builtin_amdgcn_wave_barrier();
    return {lane < n ? bench.out[lane] : 0};
}

// Adds (m, s, t) of another part to this one: what was summed under the lower maximum fades.
__device__ __forceinline__ void fade_to(float to, float m, float &s, float &t)
{
    if (s > 0.0f) {
        const float y = (m - to) * LOG2E, f = __builtin_amdgcn_exp2f(y);
        t = f > 0.0f ? f * __builtin_fmaf(y, s, t) : 0.0f;
        s *= f;
    }
}

__device__ __forceinline__ float sum_over_wave(float v)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        v += __shfl_xor(v, off, WAVE);
    return v;
}

// One wave: the list of `parts` lists of `top` keys each, in order.  Each list has
// h = ceil(top / parts) keys not below its h-th, so together they have `top` not
// below the lowest of these: that is the bound.
__device__ __forceinline__ List join_lists(const uint64_t *keys, uint32_t parts, uint32_t top, Bench &bench, uint32_t lane)
{
    const uint32_t h = (top + parts - 1) / parts;
    uint64_t bound = ~0ull;
    for (uint32_t p = lane; p < parts; p += 64)
        bound = min(bound, keys[p * top + h - 1]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        bound = min(bound, (uint64_t)__shfl_xor(bound, off, WAVE));
    constexpr int U = 8;                   // loads on their way together
    uint32_t n = 0;
    for (uint32_t i0 = 0; i0 < parts * top; i0 += 64 * U) {
        uint64_t k[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            k[u] = i0 + 64 * u + lane < parts * top ? keys[i0 + 64 * u + lane] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            n = collect(bench, n, k[u] != 0 && k[u] >= bound, k[u]);
    }
    if (n <= ROOM)
        return in_order(bench, n, lane);
    // more than there is room for (many equal logits): one after the other
    List best = {lane < top ? keys[lane] : 0};
    uint64_t least = best.at(top - 1);
    for (uint32_t i = top; i < parts * top; i += 64)
        merge(best, least, i + lane < parts * top ? keys[i + lane] : 0, top, lane);
    return best;
}

// One wave: joins `parts` results and writes the row's outputs.
template <bool F32>
__device__ __forceinline__ void finish(const LogprobArgs &a, uint32_t row, const Sums *sums, const uint64_t *keys,
                                       uint32_t parts, Bench &bench, uint32_t lane)
{
    const uint32_t target = a.targets ? (uint32_t)a.targets[row] : 0;
    float x = 0.0f;
    if (a.targets && target < a.vocab) {
        const size_t e = (size_t)row * a.vocab + target;
        x = F32 ? ((const float *)a.logits)[e] : __uint_as_float((uint32_t)((const uint16_t *)a.logits)[e] << 16);
    }
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
            a.logprob[row] = target < a.vocab ? x - base - norm : 0.0f;
        if (a.entropy)
            a.entropy[row] = s == 0.0f ? 0.0f : norm - LN2 * (t / s);
    }
    if (a.top == 0)
        return;
    const List best = join_lists(keys, parts, a.top, bench, lane);
    if (lane < a.top) {
        const uint32_t id = 0xFFFFFFFFu - (uint32_t)best.key;
        // a row with NaN may have fewer than `top` values that compare
        a.ids[(size_t)row * a.top + lane] = id < a.vocab ? (int32_t)id : 0;
        a.top_logprobs[(size_t)row * a.top + lane] =
            id < a.vocab ? from_ordered((uint32_t)(best.key >> 32)) - base - norm : __builtin_nanf("");
    }
}

// WITH_TOP: the list is kept at all; WITH_T: the entropy's sum is.
template <bool F32, bool WITH_TOP, bool WITH_T>
__global__ __launch_bounds__(WG) void k_logprobs(LogprobArgs a, uint32_t parts)
{
    constexpr int V = F32 ? 4 : 8;         // elements of 16 bytes
    constexpr uint32_t PIECE = 64 * NV * V;
    __shared__ Sums sums[WAVES];
    __shared__ uint64_t keys[WAVES * 32];
    __shared__ Bench bench[WITH_TOP ? WAVES : 1];
    const uint32_t row = blockIdx.x / parts, part = blockIdx.x % parts;
    const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t begin = row * a.vocab, end = begin + a.vocab;    // below 2^31
    const uint32_t stride = PIECE * WAVES * parts;
    uint32_t pos = begin / V * V + PIECE * (part * WAVES + wave);

    u32x4 raw[NV];
    auto load = [&](uint32_t p) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t f = p + (64 * v + lane) * V;
            if (f >= begin && f + V <= end) {
                raw[v] = *(const u32x4 *)((const uint8_t *)a.logits + (size_t)f * (F32 ? 4 : 2));
                continue;
            }
            // the row's ragged ends: only what belongs to it is read
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    raw[v][j] = f + j >= begin && f + j < end ? ((const uint32_t *)a.logits)[f + j] : 0xFF800000u;
                } else {
                    const uint32_t g = f + 2 * j;
                    const uint32_t lo = g >= begin && g < end ? ((const uint16_t *)a.logits)[g] : 0xFF80u;
                    const uint32_t hi = g + 1 >= begin && g + 1 < end ? ((const uint16_t *)a.logits)[g + 1] : 0xFF80u;
                    raw[v][j] = hi << 16 | lo;
                }
            }
        }
    };

    float m = -INFINITY, s = 0.0f, t = 0.0f;
    List best = {0};
    uint64_t least = 0;                    // what an element has to pass to enter the list
    float least_x = -INFINITY;             // its value
    bool first = true;
    if (pos < end)
        load(pos);
    for (; pos < end; pos += stride) {
        float x[NV][V], most[NV], top = -INFINITY;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    x[v][j] = __uint_as_float(raw[v][j]);
                } else {
                    x[v][2 * j % V] = bf16_lo(raw[v][j]);
                    x[v][(2 * j + 1) % V] = bf16_hi(raw[v][j]);
                }
            }
            most[v] = x[v][0];
#pragma unroll
            for (int j = 1; j < V; ++j)
                most[v] = __builtin_fmaxf(most[v], x[v][j]);
            top = __builtin_fmaxf(top, most[v]);
        }
        if (pos + stride < end)
            load(pos + stride);

        // ---- sums
        const float to = __builtin_fmaxf(m, top);
        fade_to(to, m, s, t);
        m = to;
        // x log2(e) - m log2(e) in one step where m allows it; -200 stands for all
        // that is nothing in F32, so that -inf adds 0 and not NaN to t
        if (__all(__builtin_fabsf(m) < 0x1p125f)) {
            const float by = -m * LOG2E;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float y = WITH_T ? __builtin_fmaxf(__builtin_fmaf(x[v][j], LOG2E, by), -200.0f)
                                           : __builtin_fmaf(x[v][j], LOG2E, by);
                    const float e = __builtin_amdgcn_exp2f(y);
                    s += e;
                    if (WITH_T)
                        t = __builtin_fmaf(e, y, t);
                }
        } else {
            const float by = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float y = __builtin_fmaxf((x[v][j] - by) * LOG2E, -200.0f);
                    const float e = __builtin_amdgcn_exp2f(y);
                    s += e;
                    t = __builtin_fmaf(e, y, t);
                }
        }

        // ---- the largest
        if (!WITH_TOP)
            continue;
        if (first) {
            first = false;
            // the largest value with 16 zeros behind it that `top` lanes' maxima reach
            const uint32_t u = ordered(top);
            uint32_t bound = 0;
#pragma unroll
            for (int b = 31; b >= 16; --b)
                if ((uint32_t)__popcll(__ballot(u >= (bound | 1u << b))) >= a.top)
                    bound |= 1u << b;
            // below -inf lie the keys that are no numbers
            const float bound_x = bound > ordered(-INFINITY) ? from_ordered(bound) : -INFINITY;
            uint32_t n = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!__any(most[v] >= bound_x))
                    continue;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint32_t id = pos + (64 * v + lane) * V + j - begin;
                    n = collect(bench[wave], n, x[v][j] >= bound_x && id < a.vocab,
                                (uint64_t)ordered(x[v][j]) << 32 | (0xFFFFFFFFu - id));
                }
            }
            if (n <= ROOM) {
                best = in_order(bench[wave], n, lane);
                least = best.at(a.top - 1);
                least_x = least ? from_ordered((uint32_t)(least >> 32)) : -INFINITY;
                if (least)
                    continue;
                best.key = 0;              // fewer than `top`: all over, one after the other
            }
        }
        bool touched = least == 0;         // the list has elements of this piece, which may lie behind its others
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!__any(most[v] > least_x || (touched && most[v] == least_x)))
                continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t id = pos + (64 * v + lane) * V + j - begin;
                for (uint64_t who = __ballot((x[v][j] > least_x || (touched && x[v][j] == least_x)) && id < a.vocab); who;
                     who &= who - 1) {
                    const uint32_t l = __builtin_ctzll(who);
                    const float c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x[v][j]), l));
                    const uint64_t k = (uint64_t)ordered(c) << 32 |
                                       (0xFFFFFFFFu - (uint32_t)__builtin_amdgcn_readlane(id, l));
                    if (k > least) {
                        best.insert(k, lane);
                        touched = true;
                        const uint64_t last = best.at(a.top - 1);
                        if (last > least) {
                            least = last;
                            least_x = from_ordered((uint32_t)(last >> 32));
                        }
                    }
                }
            }
        }
    }

    const float all = wave_max(m);
    fade_to(all, m, s, t);
    s = sum_over_wave(s);
    t = sum_over_wave(t);
    if (lane == 0)
        sums[wave] = {all, s, t, 0.0f};
    if (WITH_TOP && lane < a.top)
        keys[wave * a.top + lane] = best.key;
    __syncthreads();
    if (wave != 0)
        return;
    if (parts == 1) {
        finish<F32>(a, row, sums, keys, WAVES, bench[0], lane);
        return;
    }
    // the workgroup's sums and list, for the join
    float top = all;
    for (uint32_t u = 1; u < WAVES; ++u)
        top = __builtin_fmaxf(top, sums[u].m);
    fade_to(top, all, s, t);
    for (uint32_t u = 1; u < WAVES; ++u) {
        Sums p = sums[u];
        fade_to(top, p.m, p.s, p.t);
        s += p.s;
        t += p.t;
    }
    Sums *to_sums = (Sums *)a.work;
    uint64_t *to_keys = (uint64_t *)(to_sums + (size_t)a.rows * parts);
    if (lane == 0)
        to_sums[blockIdx.x] = {top, s, t, 0.0f};
    if (WITH_TOP) {
        best = join_lists(keys, WAVES, a.top, bench[0], lane);
        if (lane < a.top)
            to_keys[(size_t)blockIdx.x * a.top + lane] = best.key;
    }
}

template <bool F32>
__global__ __launch_bounds__(64) void k_logprobs_join(LogprobArgs a, uint32_t parts)
{
    __shared__ Bench bench;
    const Sums *sums = (const Sums *)a.work;
    const uint64_t *keys = (const uint64_t *)(sums + (size_t)a.rows * parts);
    const size_t first = (size_t)blockIdx.x * parts;
    finish<F32>(a, blockIdx.x, sums + first, keys + first * a.top, parts, bench, threadIdx.x);
}

// Workgroups of a row: as few as keep the chip's last round of workgroups from
// being a poor one (its rounds rounded up are then at most 1/8 more than they
// are), each wave having a piece of its own.
uint32_t parts_of(uint32_t rows, uint32_t vocab, bool f32)
{
    const uint64_t cus = cu_count() ? cu_count() : 256, piece = 64 * NV * (f32 ? 4 : 8) * WAVES;
    const uint64_t most = (vocab + piece - 1) / piece, room = 7 * cus;
    uint64_t parts = 1;
    while (parts < most && 8 * room * ((rows * parts + room - 1) / room) > 9 * rows * parts)
        ++parts;
    return (uint32_t)parts;
}

template <bool F32>
void launch(const LogprobArgs &a, hipStream_t st)
{
    const uint32_t parts = parts_of(a.rows, a.vocab, F32);
    const dim3 grid(a.rows * parts);
    if (a.top != 0 && a.entropy)
        k_logprobs<F32, true, true><<<grid, WG, 0, st>>>(a, parts);
    else if (a.top != 0)
        k_logprobs<F32, true, false><<<grid, WG, 0, st>>>(a, parts);
    else if (a.entropy)
        k_logprobs<F32, false, true><<<grid, WG, 0, st>>>(a, parts);
    else
        k_logprobs<F32, false, false><<<grid, WG, 0, st>>>(a, parts);
    count_launch();
    if (parts > 1) {
        k_logprobs_join<F32><<<a.rows, 64, 0, st>>>(a, parts);
        count_launch();
    }
}

} // namespace

uint64_t token_logprobs_work(uint32_t rows, uint32_t vocab, uint32_t top)
{
    const uint64_t parts = max(parts_of(rows, vocab, false), parts_of(rows, vocab, true));
    return parts > 1 ? (uint64_t)rows * parts * (sizeof(Sums) + 8 * top) : 16;
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

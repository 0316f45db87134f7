// prompt_short.hip -- attention over whole prompts and its gradients where there
// are few rows, for gfx950: the sums of prompt.hip and prompt_backward.hip, with
// the long axis shared out over the waves of a workgroup.
//
// A workgroup has 32 rows (or tokens) of a head, its four waves take the tiles of
// 32 on the other side in turn, each with tiles of its own in LDS (so that no
// barrier is on the way), and their sums are joined through LDS at the end, in a
// fixed order.  A short call is then four times as many workgroups, each a
// quarter as long: what bounds it is the chain from a load to the product that
// needs it, not the card's rates.  (One prompt of 301 tokens, 16 heads over 4 of
// 128 in bf16: 9.0 us, 10.5 in blocks of 128; the gradients of 2 x 150 tokens, 4
// heads over 2 of 64 in fp32: 34.5 us, 13.8 and 21.1, for 79.)  few_rows says
// where it is taken, with both sides measured.  key_kernel<float, 128> spills 38 of its
// 512 registers.
#include "prompt_internal.h"

namespace gdr {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kRows = 32;

struct KArgs {
    PromptArgs a;
    float c;              // forward: |scale| log2 e, above 0; else scale log2 e
    float ascale;         // |scale|
    bool negative;        // forward: scale < 0
    float *lse2, *start;  // [Hq, T_total]: backward (prompt_internal.h)
};

// A wave's own tiles of 32 rows of two arrays: two on their way, or one where
// two would not fit (fp32, 128 channels).
template <typename T, int D>
struct Own {
    using R = Rows<T, D>;
    static constexpr int kBytes = kRows * R::kRowBytes, kLoads = kBytes / 1024;
    static constexpr int kBufs = kBytes > 8192 ? 1 : 2;
    static constexpr int kWave = kBufs * 2 * kBytes;           // a wave's LDS
    // the join's rows: a wave's sums, 16 bytes more a row
    static constexpr int kPad = D + 4, kSums = kRows * kPad * 4;

    char *lds;
    int lane;
    __device__ inline const char *tile(int buf, int which) const {
        return lds + (2 * buf + which) * kBytes;
    }
    // rows row0 .. of a head into a tile; from `valid` (>= 1) on copies of the last
    __device__ inline void fetch(int buf, int which, const T *head, size_t row0, int valid,
                                 unsigned pitch) const {
        constexpr int kPer = 1024 / R::kRowBytes;
        const u32x4 from = source(reinterpret_cast<const char *>(head) + row0 * pitch, 0xFFFFFFFFu);
        const unsigned to = lds_address(tile(buf, which));
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int j = i * kPer + lane / R::kChunks, row = j < valid ? j : valid - 1;
            load_lds(to + 1024u * i, from, row * pitch + 16u * (lane % R::kChunks ^ R::swz(j)));
        }
    }
    // waits for the older of two tiles (LOADS of the younger one may be on
    // their way), or for all
    template <int LOADS>
    __device__ static inline void landed(bool younger) {
        static_assert(LOADS < 64, "vmcnt");
        if (younger) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(LOADS) : "memory");
        else         asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    // before a tile is fetched over one that was read
    __device__ static inline void read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
};

// One output row's channels 4 x .. of the waves' sums, joined: y = sum f_w s_w, each
// product rounded.
template <int D>
__device__ inline f32x4 join4(const char *lds, int stride, int row, int d, const float *f) {
#pragma clang fp contract(off)
    f32x4 y{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const f32x4 s = *reinterpret_cast<const f32x4 *>(lds + w * stride + (row * (D + 4) + d) * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += f[w] * s[e];
    }
    return y;
}
template <typename T> __device__ inline void store4(T *to, f32x4 y) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<bf16x4 *>(to) = cvt4(y);
    else                          *reinterpret_cast<f32x4 *>(to) = y;
}

// ------------------------------------------------------------------ forward

template <typename T, int D>
__global__ __launch_bounds__(kThreads, 1) void prompt_kernel(KArgs k) {
    using R = Rows<T, D>;
    using O = Own<T, D>;
    constexpr int kCols = R::kCols, kBufs = O::kBufs, kLds = O::kWave > O::kSums ? O::kWave : O::kSums;
    __shared__ __align__(1024) char lds[kWaves * kLds];
    __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];
    __shared__ unsigned odd_rows[kWaves];
    const PromptArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int w = uniform(tid >> 6);
    const int head = query_head(a, blockIdx.x % a.Hq);
    const Block bl = find_block<kRows, false>(a, blockIdx.x / a.Hq, 0);
    if (bl.i < 0) return;
    const int i0 = bl.i * kRows, i = i0 + r, hk = head / a.G;
    const unsigned kpitch = a.Hkv * D * (unsigned)sizeof(T);
    const T *kh = static_cast<const T *>(a.k) + (size_t)hk * D;
    const T *vh = static_cast<const T *>(a.v) + (size_t)hk * D;
    const typename R::At at = R::at(lane);
    const O own{lds + w * kLds, lane};

    const int last = i0 + kRows < bl.len ? i0 + kRows - 1 : bl.len - 1;
    const int first = a.window > 0 && i0 >= a.window ? i0 - a.window + 1 : 0;
    const int t0 = first / 32 + w, t1 = last / 32 + 1;       // this wave's: t0, t0 + 4, ..
    const unsigned span = a.window > 0 ? a.window : 1u << 31;
    auto attends = [&](int j) GDR_INLINE { return (unsigned)(i - j) < span; };
    auto tile_full = [&](int t) GDR_INLINE {
        return t * 32 + 31 <= i0 && (a.window == 0 || t * 32 > i0 + 31 - a.window);
    };
    auto stage = [&](int t, int buf) GDR_INLINE {
        const size_t row = (size_t)bl.row0 + t * 32;
        const int left = bl.len - t * 32;
        own.fetch(buf, 0, kh, row, left, kpitch);
        own.fetch(buf, 1, vh, row, left, kpitch);
    };
    typename R::B q;
    float m, mc, l, down = 1.f;
    unsigned small = 0;                      // rows whose weights are kDown times theirs
    f32x16 acc[kCols];
    auto walk = [&](auto clear) GDR_INLINE {
        constexpr bool CLEAR = decltype(clear)::value;
        m = -INFINITY;
        mc = l = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c][e] = 0.f;
        if (!CLEAR) {
            const int row = i < bl.len ? i : bl.len - 1;
            R::load(q, static_cast<const T *>(a.q) + ((size_t)(bl.row0 + row) * a.Hq + head) * D, h);
        }
        if (t0 < t1) stage(t0, 0);
        if (kBufs > 1 && t0 + kWaves < t1) stage(t0 + kWaves, 1);
        R::settle(q);
        if (!CLEAR && k.negative) R::negate(q);
        int buf = 0;
        for (int t = t0; t < t1; t += kWaves) {
            O::template landed<2 * O::kLoads>(kBufs > 1 && t + kWaves < t1);
            f32x16 x = R::rows(own.tile(buf, 0), 0, at, q);
            const bool full = tile_full(t);
            if (!full) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = attends(t * 32 + R::key(e, h)) ? x[e] : -INFINITY;
            }
            float top = x[0];
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, x[e]);
            const float mn = fmaxf(m, swap_max32(top));
            const bool grow = (mn - m) * k.c > 8.f;
            if (__builtin_amdgcn_ballot_w64(grow)) {
                const float al = grow ? exp2_((m - mn) * k.c) : 1.f;
                l *= al;
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[c] *= al;
                m = grow ? mn : m;
                mc = grow ? mn * k.c : mc;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[e] = exp2_(fmaf(x[e], k.c, -mc));
                if (CLEAR) x[e] *= down;
                l += x[e];
            }
            R::template cols<CLEAR>(acc, own.tile(buf, 1), 0, at, R::operand(x), full);
            O::read();
            if (t + kBufs * kWaves < t1) stage(t + kBufs * kWaves, buf);
            if (kBufs > 1) buf ^= 1;
        }
    };
    walk(std::false_type{});
    if (__builtin_expect(__syncthreads_or(R::any_odd(acc)), 0)) {
        // (as in prompt.hip, the rows to be smaller those of any wave)
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            walk(std::true_type{});
            if (pass) break;
            const unsigned odd = rows_of(R::any_odd(acc));
            if (lane == 0) odd_rows[w] = odd;
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kWaves; ++u) small |= odd_rows[u];
            if (!small) break;
            down = small >> r & 1 ? kDown : 1.f;
        }
        for (int t = t0; t < t1; t += kWaves)
            for (int j = t * 32; j < t * 32 + 32 && j <= last; ++j)
                if (!tile_full(t) && attends(j))
                    R::add_odd(acc, vh + (size_t)(bl.row0 + j) * a.Hkv * D, h);
    }
    l = swap_sum32(l);
    if (h == 0) {
        sm[w][r] = m;
        sl[w][r] = l;
    }
    R::put(reinterpret_cast<float *>(own.lds) + r * O::kPad, acc, h);
    __syncthreads();
    // eight threads a row
    const int row = tid / 8, x = tid % 8;
    if (i0 + row >= bl.len) return;
    float top = -INFINITY, f[kWaves], sum = 0.f;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) top = fmaxf(top, sm[u][row]);
    // A wave whose tokens the row does not attend to has m = -inf, f = 0 and sums of
    // zero.  So has, but for its sums, one whose logits are all NaN, which the maximum
    // passes over: 0 times these are NaN.
    const float ms = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int u = 0; u < kWaves; ++u) {
#pragma clang fp contract(off)
        f[u] = exp2_((sm[u][row] - ms) * k.c);
        sum += sl[u][row] * f[u];
    }
    const size_t to = (size_t)(bl.row0 + i0 + row) * a.Hq + head;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int d = 4 * x; d < D; d += 32) {
        f32x4 y = join4<D>(lds, kLds, row, d, f) * inv;
        if (sum == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
        // (finite sums of the waves may add up to an infinity)
        if (!(fabsf(y[0]) < INFINITY & fabsf(y[1]) < INFINITY & fabsf(y[2]) < INFINITY &
              fabsf(y[3]) < INFINITY)) {
            float g[kWaves];
#pragma unroll
            for (int u = 0; u < kWaves; ++u) g[u] = f[u] * inv;
            const f32x4 z = join4<D>(lds, kLds, row, d, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = fabsf(y[e]) < INFINITY ? y[e] : z[e];
        }
        store4(static_cast<T *>(a.o) + to * D + d, y);
    }
    if (a.lse && x == 0)
        a.lse[to] = sum == 0.f ? -INFINITY
                               : ms * k.ascale + kLn2F * __builtin_amdgcn_logf(
                                                             small >> row & 1 ? sum * kUp : sum);
}

// ------------------------------------------------------------------ backward

template <typename T, int D>
__global__ __launch_bounds__(kThreads, 1) void query_kernel(KArgs k) {
    using R = Rows<T, D>;
    using O = Own<T, D>;
    constexpr int kCols = R::kCols, kBufs = O::kBufs, kLds = O::kWave > O::kSums ? O::kWave : O::kSums;
    __shared__ __align__(1024) char lds[kWaves * kLds];
    const PromptArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int w = uniform(tid >> 6);
    const int head = query_head(a, blockIdx.x % a.Hq);
    const Block bl = find_block<kRows, false>(a, blockIdx.x / a.Hq, 0);
    if (bl.i < 0) return;
    const int i0 = bl.i * kRows, i = i0 + r, hk = head / a.G;
    const unsigned kpitch = a.Hkv * D * (unsigned)sizeof(T);
    const T *kh = static_cast<const T *>(a.k) + (size_t)hk * D;
    const T *vh = static_cast<const T *>(a.v) + (size_t)hk * D;
    const typename R::At at = R::at(lane);
    const O own{lds + w * kLds, lane};
    const int last = i0 + kRows < bl.len ? i0 + kRows - 1 : bl.len - 1;
    const int first = a.window > 0 && i0 >= a.window ? i0 - a.window + 1 : 0;
    const int t0 = first / 32 + w, t1 = last / 32 + 1;
    const unsigned span = a.window > 0 ? a.window : 1u << 31;
    auto attends = [&](int j) GDR_INLINE { return (unsigned)(i - j) < span; };
    auto stage = [&](int t, int buf) GDR_INLINE {
        const size_t row = (size_t)bl.row0 + t * 32;
        const int left = bl.len - t * 32;
        own.fetch(buf, 0, kh, row, left, kpitch);
        own.fetch(buf, 1, vh, row, left, kpitch);
    };
    typename R::B q, g;
    float lse2, start;
    f32x16 acc[kCols];
    auto walk = [&](auto clear) GDR_INLINE {
        constexpr bool CLEAR = decltype(clear)::value;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c][e] = 0.f;
        if (t0 < t1) stage(t0, 0);
        if (kBufs > 1 && t0 + kWaves < t1) stage(t0 + kWaves, 1);
        if (!CLEAR) {
            const int row = bl.row0 + (i < bl.len ? i : bl.len - 1);
            const size_t at_row = ((size_t)row * a.Hq + head) * D;
            R::load(q, static_cast<const T *>(a.q) + at_row, h);
            R::load(g, static_cast<const T *>(a.d_o) + at_row, h);
            lse2 = base2(a.lse[(size_t)row * a.Hq + head]);
            start = minus_delta<T, D>(static_cast<const T *>(a.d_o) + at_row,
                                    static_cast<const T *>(a.o) + at_row, h);
            if (i < bl.len && h == 0 && w == 0) {
                k.lse2[(size_t)head * a.T_total + row] = lse2;
                k.start[(size_t)head * a.T_total + row] = start;
            }
        }
        R::settle(q);
        R::settle(g);
        asm volatile("" : "+v"(lse2));
        f32x16 from;
#pragma unroll
        for (int e = 0; e < 16; ++e) from[e] = start;
        asm volatile("" : "+v"(from));
        int buf = 0;
        for (int t = t0; t < t1; t += kWaves) {
            O::template landed<2 * O::kLoads>(kBufs > 1 && t + kWaves < t1);
            const bool full = t * 32 + 31 <= i0 && (a.window == 0 || t * 32 > i0 + 31 - a.window);
            f32x16 x = R::rows(own.tile(buf, 0), 0, at, q);
            const f32x16 dp = R::rows(own.tile(buf, 1), 0, at, g, from);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = exp2_(fmaf(x[e], k.c, -lse2)) * dp[e];
            if (!full) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = attends(t * 32 + R::key(e, h)) ? x[e] : 0.f;
            }
            R::template cols<CLEAR>(acc, own.tile(buf, 0), 0, at, R::operand(x), full);
            O::read();
            if (t + kBufs * kWaves < t1) stage(t + kBufs * kWaves, buf);
            if (kBufs > 1) buf ^= 1;
        }
    };
    walk(std::false_type{});
    if (__builtin_expect(__syncthreads_or(R::any_odd(acc)), 0)) walk(std::true_type{});
    R::put(reinterpret_cast<float *>(own.lds) + r * O::kPad, acc, h);
    __syncthreads();
    const int row = tid / 8, x = tid % 8;
    if (i0 + row >= bl.len) return;
    const float one[kWaves] = {1.f, 1.f, 1.f, 1.f};
    T *to = static_cast<T *>(a.dq) + ((size_t)(bl.row0 + i0 + row) * a.Hq + head) * D;
#pragma unroll
    for (int d = 4 * x; d < D; d += 32) store4(to + d, join4<D>(lds, kLds, row, d, one) * a.scale);
}

// Workgroup = (block of 32 tokens, key-value head); the waves take the tiles of
// rows of all heads of the group in turn.
template <typename T, int D>
__global__ __launch_bounds__(kThreads, 1) void key_kernel(KArgs k) {
    using R = Rows<T, D>;
    using O = Own<T, D>;
    constexpr int kCols = R::kCols, kBufs = O::kBufs;
    constexpr int kLds = O::kWave > 2 * O::kSums ? O::kWave : 2 * O::kSums;
    __shared__ __align__(1024) char lds[kWaves * kLds];
    __shared__ __align__(16) float stats[kWaves][kBufs][2][32];    // lse2 and -delta of a tile's rows
    const PromptArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int w = uniform(tid >> 6);
    const int hk = blockIdx.x % a.Hkv;
    const Block bl = find_block<kRows, true>(a, blockIdx.x / a.Hkv, 0);
    if (bl.i < 0) return;
    const int j0 = bl.i * kRows, j = j0 + r;
    const unsigned qpitch = a.Hq * D * (unsigned)sizeof(T);
    const typename R::At at = R::at(lane);
    const O own{lds + w * kLds, lane};
    const unsigned span = a.window > 0 ? a.window : 1u << 31;
    const int over = a.window > 0 && bl.len - j0 > kRows + a.window - 1 ? j0 + kRows + a.window - 1
                                                                         : bl.len;
    const int t0 = j0 / 32, tiles = (over - 1) / 32 + 1 - t0, all = tiles * a.G;
    auto stage = [&](int n, int buf) GDR_INLINE {
        const int head = hk * a.G + n / tiles, t = t0 + n % tiles, left = bl.len - t * 32;
        const size_t first = (size_t)bl.row0 + t * 32;
        own.fetch(buf, 0, static_cast<const T *>(a.q) + (size_t)head * D, first, left, qpitch);
        own.fetch(buf, 1, static_cast<const T *>(a.d_o) + (size_t)head * D, first, left, qpitch);
        const int at_row = r < left ? r : left - 1;
        const size_t from = (size_t)head * a.T_total + first;
        fetch_words<32>(stats[w][buf][0], k.lse2 + from, at_row, lane);
        fetch_words<32>(stats[w][buf][1], k.start + from, at_row, lane);
    };
    typename R::B kf, vf;
    f32x16 dk[kCols], dv[kCols];
    auto walk = [&](auto clear) GDR_INLINE {
        constexpr bool CLEAR = decltype(clear)::value;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) dk[c][e] = dv[c][e] = 0.f;
        if (w < all) stage(w, 0);
        if (kBufs > 1 && w + kWaves < all) stage(w + kWaves, 1);
        if (!CLEAR) {
            const int row = bl.row0 + (j < bl.len ? j : bl.len - 1);
            R::load(kf, static_cast<const T *>(a.k) + ((size_t)row * a.Hkv + hk) * D, h);
            R::load(vf, static_cast<const T *>(a.v) + ((size_t)row * a.Hkv + hk) * D, h);
        }
        R::settle(kf);
        R::settle(vf);
        int buf = 0;
        for (int n = w; n < all; n += kWaves) {
            O::template landed<2 * O::kLoads + 2>(kBufs > 1 && n + kWaves < all);
            const int i0 = (t0 + n % tiles) * 32;
            const bool full = i0 >= j0 + 31 && i0 + 32 <= bl.len &&
                              (a.window == 0 || i0 + 31 < j0 + a.window);
            const float *lse2 = stats[w][buf][0], *start = stats[w][buf][1];
            f32x16 x = R::rows(own.tile(buf, 0), 0, at, kf);
            f32x16 dp = R::rows(own.tile(buf, 1), 0, at, vf, R::per_row(start, h));
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const f32x4 ls = *reinterpret_cast<const f32x4 *>(lse2 + R::key(e, h));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    x[e + u] = exp2_(fmaf(x[e + u], k.c, -ls[u]));
                    dp[e + u] *= x[e + u];
                }
            }
            if (!full) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = i0 + R::key(e, h);
                    const bool in = (unsigned)(i - j) < span & i < bl.len;
                    x[e] = in ? x[e] : 0.f;
                    dp[e] = in ? dp[e] : 0.f;
                }
            }
            R::template cols<CLEAR>(dv, own.tile(buf, 1), 0, at, R::operand(x), full);
            R::template cols<CLEAR>(dk, own.tile(buf, 0), 0, at, R::operand(dp), full);
            O::read();
            if (n + kBufs * kWaves < all) stage(n + kBufs * kWaves, buf);
            if (kBufs > 1) buf ^= 1;
        }
    };
    walk(std::false_type{});
    if (__builtin_expect(__syncthreads_or(R::any_odd(dk) || R::any_odd(dv)), 0))
        walk(std::true_type{});
    R::put(reinterpret_cast<float *>(own.lds) + r * O::kPad, dk, h);
    R::put(reinterpret_cast<float *>(own.lds + O::kSums) + r * O::kPad, dv, h);
    __syncthreads();
    const int row = tid / 8, x = tid % 8;
    if (j0 + row >= bl.len) return;
    const float one[kWaves] = {1.f, 1.f, 1.f, 1.f};
    const size_t to = ((size_t)(bl.row0 + j0 + row) * a.Hkv + hk) * D;
#pragma unroll
    for (int d = 4 * x; d < D; d += 32) {
        store4(static_cast<T *>(a.dk) + to + d, join4<D>(lds, kLds, row, d, one) * a.scale);
        store4(static_cast<T *>(a.dv) + to + d, join4<D>(lds + O::kSums, kLds, row, d, one));
    }
}

template <typename T, int D>
hipError_t forward(const PromptArgs &a, hipStream_t s) {
    KArgs k{};
    k.a = a;
    k.ascale = fabsf(a.scale);
    k.c = fminf(fmaxf(fabsf(a.scale * kLog2e), 1.4e-45f), 3.4e38f);
    k.negative = a.scale < 0.f;
    prompt_kernel<T, D><<<(unsigned)(block_bound<kRows>(a) * a.Hq), kThreads, 0, s>>>(k);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t backward_q(const PromptArgs &a, hipStream_t s) {
    KArgs k{};
    k.a = a;
    k.c = fminf(fmaxf(a.scale * kLog2e, -3.4e38f), 3.4e38f);
    k.lse2 = static_cast<float *>(a.ws);
    k.start = k.lse2 + (size_t)a.Hq * a.T_total;
    query_kernel<T, D><<<(unsigned)(block_bound<kRows>(a) * a.Hq), kThreads, 0, s>>>(k);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t backward_k(const PromptArgs &a, hipStream_t s) {
    KArgs k{};
    k.a = a;
    k.c = fminf(fmaxf(a.scale * kLog2e, -3.4e38f), 3.4e38f);
    k.lse2 = static_cast<float *>(a.ws);
    k.start = k.lse2 + (size_t)a.Hq * a.T_total;
    key_kernel<T, D><<<(unsigned)(block_bound<kRows>(a) * a.Hkv), kThreads, 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_short(bool bf16_io, int D, const PromptArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? forward<bf16, 128>(a, s) : forward<bf16, 64>(a, s);
    return D == 128 ? forward<float, 128>(a, s) : forward<float, 64>(a, s);
}
hipError_t launch_queries_short(bool bf16_io, int D, const PromptArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? backward_q<bf16, 128>(a, s) : backward_q<bf16, 64>(a, s);
    return D == 128 ? backward_q<float, 128>(a, s) : backward_q<float, 64>(a, s);
}
hipError_t launch_keys_short(bool bf16_io, int D, const PromptArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? backward_k<bf16, 128>(a, s) : backward_k<bf16, 64>(a, s);
    return D == 128 ? backward_k<float, 128>(a, s) : backward_k<float, 64>(a, s);
}

}  // namespace gdr

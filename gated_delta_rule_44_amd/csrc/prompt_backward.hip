// prompt_backward.hip -- the gradients of attention over whole prompts, for
// gfx950.
//
// With s_ij = scale q_i.k_j, w_ij = e^{s_ij - lse_i}, delta_i = do_i.o_i:
//     ds_ij = w_ij (do_i.v_j - delta_i),
//     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
//     dv_j = sum_i w_ij do_i.
//
// Two kernels, so that no sum is shared between workgroups: query_kernel walks
// a block of rows over its tokens (s, do.v and dq: three products), key_kernel
// a block of tokens over the rows of every head of its group that attend to
// it (s, do.v, dv and dk: four).  Seven products where five would do, for
// results that do not depend on the order of workgroups.
//
// Products bound it.  4 sequences of 4,096 tokens, 32 heads over 8 of 128 in bf16:
// 1,850 to 1,967 us, query_kernel 790 (1.04 PFLOP/s) and key_pairs_kernel 1,120
// (0.98), the matrix units busy for 55 and 50 % of the CUs' cycles; the floor of
// seven products at a library's rate is 1,582.  12 packed sequences of 300 to 6,100
// tokens, window 512, 16 heads of 64: 307 to 332 us, 137 and 195, busy for 34 and
// 28 %: of 64 channels the exponentials and what is done to ds take as long as the
// products, and a sixth of what a wave's tiles hold is masked.  fp32 has a kernel for
// the keys that is one wave a SIMD (its accumulators fill the registers).
//   key_pairs_kernel<128, 4> spills 36 registers (100 bytes a lane): some 38 MB of the
// 105 MB that the first case is seen to write; one tile loop loads five of them again.
#include "prompt_internal.h"

namespace gdr {
namespace {

constexpr int kWaves = 4;                  // waves of a workgroup, 32 rows or tokens each
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;

// Workspace: lse log2 e (+inf for a row without weights) and -delta of every
// row, head by head.  The sums do.v start from -delta, so that none is taken off
// after them (4 x 4,096 tokens 1,904 -> 1,874 us, of 64 channels 1,053 -> 1,027).
struct KArgs {
    PromptArgs a;
    float c;              // scale log2 e
    int mixed;            // mixed_seqs
    float *lse2, *start;  // [Hq, T_total]
};

// Workgroup = (block of 128 rows, query head), 32 rows a wave.
template <typename T, int D>
__global__ __launch_bounds__(kThreads, (Rows<T, D>::kRowBytes > 256 ? 1 : 2)) void query_kernel(KArgs k) {
    using R = Rows<T, D>;
    constexpr int kTok = R::kTok, kBlk = kTok / 32, kCols = R::kCols;
    __shared__ __align__(1024) char lds[2][2][R::kTileBytes];
    const PromptArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int w = uniform(tid >> 6);
    const int head = query_head(a, blockIdx.x % a.Hq);
    const Block bl = find_block<kRows, false>(a, blockIdx.x / a.Hq, k.mixed);
    if (bl.i < 0) return;
    const int i0 = bl.i * kRows, iw = i0 + 32 * w, i = iw + r;
    const int hk = head / a.G;
    const unsigned kpitch = a.Hkv * D * (unsigned)sizeof(T);
    const T *kh = static_cast<const T *>(a.k) + (size_t)hk * D;
    const T *vh = static_cast<const T *>(a.v) + (size_t)hk * D;
    const typename R::At at = R::at(lane);

    typename R::B q, g;
    float lse2, start;
    {
        const int row = bl.row0 + (i < bl.len ? i : bl.len - 1);
        const size_t at_row = ((size_t)row * a.Hq + head) * D;
        R::load(q, static_cast<const T *>(a.q) + at_row, h);
        R::load(g, static_cast<const T *>(a.d_o) + at_row, h);
        lse2 = base2(a.lse[(size_t)row * a.Hq + head]);
        start = minus_delta<T, D>(static_cast<const T *>(a.d_o) + at_row,
                                static_cast<const T *>(a.o) + at_row, h);
        if (i < bl.len && h == 0) {
            k.lse2[(size_t)head * a.T_total + row] = lse2;
            k.start[(size_t)head * a.T_total + row] = start;
        }
    }
    const int last = i0 + kRows < bl.len ? i0 + kRows - 1 : bl.len - 1;
    const int first = a.window > 0 && i0 >= a.window ? i0 - a.window + 1 : 0;
    const int t0 = first / kTok, t1 = last / kTok + 1;
    const unsigned span = a.window > 0 ? a.window : 1u << 31;     // tokens a row attends to
    auto attends = [&](int j) GDR_INLINE { return (unsigned)(i - j) < span; };
    const Fetch<T, D, kWaves> fetch(kpitch, w, lane);
    auto stage = [&](int t) GDR_INLINE {
        const size_t row = (size_t)bl.row0 + t * kTok;
        const int left = bl.len - t * kTok;
        fetch(lds[t & 1][0], kh, row, left, lane);
        fetch(lds[t & 1][1], vh, row, left, lane);
    };
    f32x16 acc[kCols];
    auto walk = [&](auto clear) GDR_INLINE {
        constexpr bool CLEAR = decltype(clear)::value;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c][e] = 0.f;
        stage(t0);
        R::settle(q);
        R::settle(g);
        asm volatile("" : "+v"(lse2));
        f32x16 from;
#pragma unroll
        for (int e = 0; e < 16; ++e) from[e] = start;
        asm volatile("" : "+v"(from));
        for (int t = t0; t < t1; ++t) {
            tile_landed();
            if (t + 1 < t1) stage(t + 1);
            const int j0 = t * kTok;
            const char *kt = lds[t & 1][0], *vt = lds[t & 1][1];
            if (iw >= bl.len || j0 > iw + 31 || (a.window > 0 && j0 + kTok <= iw - a.window + 1))
                continue;
            const bool full = j0 + kTok - 1 <= iw && (a.window == 0 || j0 > iw + 31 - a.window);
#pragma unroll
            for (int b = 0; b < kBlk; ++b) {
                f32x16 x = R::rows(kt, b, at, q);
                const f32x16 dp = R::rows(vt, b, at, g, from);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = exp2_(fmaf(x[e], k.c, -lse2)) * dp[e];
                if (!full) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[e] = attends(j0 + 32 * b + R::key(e, h)) ? x[e] : 0.f;
                }
                R::template cols<CLEAR>(acc, kt, b, at, R::operand(x), full);
            }
        }
    };
    walk(std::false_type{});
    // (0 times an infinity or NaN of a key that a row does not attend to: again
    // without those)
    if (__builtin_expect(__syncthreads_or(R::any_odd(acc)), 0)) walk(std::true_type{});
    if (i >= bl.len) return;
    R::store(static_cast<T *>(a.dq) + ((size_t)(bl.row0 + i) * a.Hq + head) * D, acc, h, a.scale);
}

// Workgroup = (block of 128 tokens, key-value head), 32 tokens a wave: lane
// (h, r) has token r of them as a column, tiles of rows pass through LDS.
template <typename T, int D>
__global__ __launch_bounds__(kThreads, 1) void key_kernel(KArgs k) {
    using R = Rows<T, D>;
    constexpr int kTok = R::kTok, kBlk = kTok / 32, kCols = R::kCols;
    __shared__ __align__(1024) char lds[2][2][R::kTileBytes];
    __shared__ __align__(16) float stats[2][2][kTok];      // lse2 and -delta of a tile's rows
    const PromptArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int w = uniform(tid >> 6);
    const int hk = blockIdx.x % a.Hkv;
    const Block bl = find_block<kRows, true>(a, blockIdx.x / a.Hkv, k.mixed);
    if (bl.i < 0) return;
    const int j0 = bl.i * kRows, jw = j0 + 32 * w, j = jw + r;
    const unsigned qpitch = a.Hq * D * (unsigned)sizeof(T);
    const typename R::At at = R::at(lane);

    typename R::B kf, vf;
    const int row = bl.row0 + (j < bl.len ? j : bl.len - 1);
    R::load(kf, static_cast<const T *>(a.k) + ((size_t)row * a.Hkv + hk) * D, h);
    R::load(vf, static_cast<const T *>(a.v) + ((size_t)row * a.Hkv + hk) * D, h);
    // rows that attend to a token of the block
    const unsigned span = a.window > 0 ? a.window : 1u << 31;     // tokens a row attends to
    const int over = a.window > 0 && bl.len - j0 > kRows + a.window - 1 ? j0 + kRows + a.window - 1
                                                                         : bl.len;
    const int t0 = j0 / kTok, tiles = (over - 1) / kTok + 1 - t0, all = tiles * a.G;

    const Fetch<T, D, kWaves> fetch(qpitch, w, lane);
    // the tiles in their order, head by head: where the next to be fetched is
    const int t1 = t0 + tiles;
    int next_head, next_t;
    auto stage = [&](int buf) GDR_INLINE {
        const int left = bl.len - next_t * kTok;
        const size_t first = (size_t)bl.row0 + next_t * kTok;
        fetch(lds[buf][0], static_cast<const T *>(a.q) + (size_t)next_head * D, first, left, lane);
        fetch(lds[buf][1], static_cast<const T *>(a.d_o) + (size_t)next_head * D, first, left, lane);
        if (w < 2)
            fetch_words<kTok>(stats[buf][w],
                              (w ? k.start : k.lse2) + (size_t)next_head * a.T_total + first,
                              lane < left ? lane : left - 1, lane);
        if (++next_t == t1) {
            next_t = t0;
            ++next_head;
        }
    };
    f32x16 dk[kCols], dv[kCols];
    auto walk = [&](auto clear) GDR_INLINE {
        constexpr bool CLEAR = decltype(clear)::value;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) dk[c][e] = dv[c][e] = 0.f;
        next_head = hk * a.G;
        next_t = t0;
        stage(0);
        R::settle(kf);
        R::settle(vf);
        for (int n = 0, t = t0; n < all; ++n) {
            tile_landed();
            if (n + 1 < all) stage((n + 1) & 1);
            const int i0 = t * kTok;
            t = t + 1 == t1 ? t0 : t + 1;
            const char *qt = lds[n & 1][0], *gt = lds[n & 1][1];
            const float *lse2 = stats[n & 1][0], *start = stats[n & 1][1];
            if (jw >= bl.len || i0 + kTok <= jw || (a.window > 0 && i0 >= jw + 31 + a.window)) continue;
            const bool full = i0 >= jw + 31 && i0 + kTok <= bl.len &&
                              (a.window == 0 || i0 + kTok - 1 < jw + a.window);
#pragma unroll
            for (int b = 0; b < kBlk; ++b) {
                f32x16 x = R::rows(qt, b, at, kf);
                f32x16 dp = R::rows(gt, b, at, vf, R::per_row(start + 32 * b, h));
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f32x4 ls = *reinterpret_cast<const f32x4 *>(lse2 + 32 * b + R::key(e, h));
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        x[e + u] = exp2_(fmaf(x[e + u], k.c, -ls[u]));
                        dp[e + u] *= x[e + u];
                    }
                }
                if (!full) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int i = i0 + 32 * b + R::key(e, h);
                        const bool in = (unsigned)(i - j) < span & i < bl.len;
                        x[e] = in ? x[e] : 0.f;
                        dp[e] = in ? dp[e] : 0.f;
                    }
                }
                R::template cols<CLEAR>(dv, gt, b, at, R::operand(x), full);
                R::template cols<CLEAR>(dk, qt, b, at, R::operand(dp), full);
            }
        }
    };
    walk(std::false_type{});
    if (__builtin_expect(__syncthreads_or(R::any_odd(dk) || R::any_odd(dv)), 0))
        walk(std::true_type{});
    if (j >= bl.len) return;
    const size_t to = ((size_t)(bl.row0 + j) * a.Hkv + hk) * D;
    R::store(static_cast<T *>(a.dk) + to, dk, h, a.scale);
    R::store(static_cast<T *>(a.dv) + to, dv, h, 1.f);
}

// The same in bf16, by pairs of waves: both waves of a pair hold the same 32
// tokens' k and v, each forms w and ds for one half of a tile's 64 rows, and
// one of them sums dv, the other dk, over all 64; what a wave has for the other
// one (w or ds of its half) passes through LDS as the operand that it is.  A
// wave then has 64 accumulators instead of 128, and two waves share a SIMD:
// one's exponentials run under the other's products.  A tile's sums are formed
// while the next one's w and ds are, so that one barrier a tile orders all.
// (4 sequences of 4,096 tokens, 128 channels: 1,824 us by one wave a SIMD, 1,308
// by pairs, 1,172 with the pair's two waves in opposite order, 1,128 as it is.)
template <int D, int PAIRS>
__global__ __launch_bounds__(128 * PAIRS, 2) void key_pairs_kernel(KArgs k) {
    typedef bf16 T;
    using R = Rows<T, D>;
    constexpr int kTok = R::kTok, kCols = R::kCols, kTokens = 32 * PAIRS;
    static_assert(kTok == 64, "a half of the rows each");
    __shared__ __align__(1024) char lds[3][2][R::kTileBytes];
    __shared__ __align__(16) bf16x8 given[2][2][PAIRS][2][64];   // [n & 1][role][pair]
    __shared__ __align__(16) float stats[3][2][kTok];
    const PromptArgs &a = k.a;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int w = uniform(tid >> 6), pair = w % PAIRS, role = w / PAIRS;
    const int hk = blockIdx.x % a.Hkv;
    const Block bl = find_block<kTokens, true>(a, blockIdx.x / a.Hkv, k.mixed);
    if (bl.i < 0) return;
    const int j0 = bl.i * kTokens, jw = j0 + 32 * pair, j = jw + r;
    const unsigned qpitch = a.Hq * D * (unsigned)sizeof(T);
    const typename R::At at = R::at(lane);

    typename R::B kf, vf;
    const int row = bl.row0 + (j < bl.len ? j : bl.len - 1);
    R::load(kf, static_cast<const T *>(a.k) + ((size_t)row * a.Hkv + hk) * D, h);
    R::load(vf, static_cast<const T *>(a.v) + ((size_t)row * a.Hkv + hk) * D, h);
    const unsigned span = a.window > 0 ? a.window : 1u << 31;     // tokens a row attends to
    const int over = a.window > 0 && bl.len - j0 > kTokens + a.window - 1 ? j0 + kTokens + a.window - 1
                                                                         : bl.len;
    const int t0 = j0 / kTok, tiles = (over - 1) / kTok + 1 - t0, all = tiles * a.G;

    const Fetch<T, D, 2 * PAIRS> fetch(qpitch, w, lane);
    // the tiles in their order, head by head: where the next to be fetched is
    const int t1 = t0 + tiles;
    int next_head, next_t;
    auto stage = [&](int buf) GDR_INLINE {
        const int left = bl.len - next_t * kTok;
        const size_t first = (size_t)bl.row0 + next_t * kTok;
        fetch(lds[buf][0], static_cast<const T *>(a.q) + (size_t)next_head * D, first, left, lane);
        fetch(lds[buf][1], static_cast<const T *>(a.d_o) + (size_t)next_head * D, first, left, lane);
        if (w < 2)
            fetch_words<kTok>(stats[buf][w],
                              (w ? k.start : k.lse2) + (size_t)next_head * a.T_total + first,
                              lane < left ? lane : left - 1, lane);
        if (++next_t == t1) {
            next_t = t0;
            ++next_head;
        }
    };
    f32x16 acc[kCols];
    typename R::P kept;                      // this wave's half of tile n, for its own sums
    // each of 32 rows from i on attends to all of the pair's tokens
    auto whole = [&](int i) GDR_INLINE {
        return i >= jw + 31 && i + 32 <= bl.len && (a.window == 0 || i + 31 < jw + a.window);
    };
    // A tile: its number in the sequence, its place in LDS and in turn of two.
    struct Tile { int t, buf, turn; };
    auto after = [&](Tile x) GDR_INLINE {
        return Tile{x.t + 1 == t1 ? t0 : x.t + 1, x.buf == 2 ? 0 : x.buf + 1, x.turn ^ 1};
    };
    // w and ds of this wave's half of a tile
    auto weights = [&](Tile n, auto which, auto between) GDR_INLINE {
        constexpr int ROLE = decltype(which)::value;
        const int i0 = n.t * kTok + 32 * ROLE;
        const char *qt = lds[n.buf][0] + 32 * ROLE * R::kRowBytes, *gt = qt + R::kTileBytes;
        const float *lse2 = stats[n.buf][0] + 32 * ROLE, *start = lse2 + kTok;
        f32x16 x = R::rows(qt, 0, at, kf);
        __builtin_amdgcn_sched_barrier(0);
        f32x16 dp = R::rows(gt, 0, at, vf, R::per_row(start, h));
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const f32x4 ls = *reinterpret_cast<const f32x4 *>(lse2 + R::key(e, h));
#pragma unroll
            for (int u = 0; u < 4; ++u) x[e + u] = exp2_(fmaf(x[e + u], k.c, -ls[u]));
        }
        __builtin_amdgcn_sched_barrier(0);
        between();
        dp *= x;
        if (!whole(i0)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = i0 + R::key(e, h);
                const bool in = (unsigned)(i - j) < span & i < bl.len;
                x[e] = in ? x[e] : 0.f;
                dp[e] = in ? dp[e] : 0.f;
            }
        }
        const typename R::P p = R::operand(x), ds = R::operand(dp);
        kept = ROLE ? ds : p;
#pragma unroll
        for (int u = 0; u < 2; ++u) given[n.turn][ROLE][pair][u][lane] = ROLE ? p.f[u] : ds.f[u];
    };
    // dv (role 0) or dk (role 1) of a tile, by this wave's half of it (mine) or
    // the other's
    auto sums = [&](Tile n, auto which, auto clear, const typename R::P &mine) GDR_INLINE {
        constexpr int ROLE = decltype(which)::value;
        const bool all = whole(n.t * kTok + 32 * ROLE);
        R::template cols<decltype(clear)::value>(
            acc, lds[n.buf][1 - ROLE] + 32 * ROLE * R::kRowBytes, 0, at, mine, all);
    };
    auto other_sums = [&](Tile n, auto which, auto clear) GDR_INLINE {
        constexpr int ROLE = decltype(which)::value;
        const bool all = whole(n.t * kTok + 32 * (1 - ROLE));
        typename R::P p;
#pragma unroll
        for (int u = 0; u < 2; ++u) p.f[u] = given[n.turn][1 - ROLE][pair][u][lane];
        R::template cols<decltype(clear)::value>(
            acc, lds[n.buf][1 - ROLE] + 32 * (1 - ROLE) * R::kRowBytes, 0, at, p, all);
    };
    // Role 0 forms its weights first and then its sums, role 1 the other way
    // round: the two waves of a SIMD are then in different parts of a tile.
    auto walk_as = [&](auto which, auto clear) GDR_INLINE {
        constexpr int ROLE = decltype(which)::value;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c][e] = 0.f;
        next_head = hk * a.G;
        next_t = t0;
        stage(0);
        R::settle(kf);
        R::settle(vf);
        tile_landed();
        if (all > 1) stage(1);
        Tile now{t0, 0, 0};
        weights(now, which, []() {});
        for (int n = 1; n < all; ++n) {
            const Tile was = now;
            now = after(now);
            tile_landed();
            if (n + 1 < all) stage(now.buf == 2 ? 0 : now.buf + 1);
            if constexpr (ROLE == 0) {
                const typename R::P mine = kept;
                weights(now, which, [&]() { sums(was, which, clear, mine); });
                __builtin_amdgcn_sched_barrier(0);
                other_sums(was, which, clear);
            } else {
                sums(was, which, clear, kept);
                __builtin_amdgcn_sched_barrier(0);
                other_sums(was, which, clear);
                __builtin_amdgcn_sched_barrier(0);
                weights(now, which, []() {});
            }
        }
        __syncthreads();
        sums(now, which, clear, kept);
        other_sums(now, which, clear);
    };
    auto walk = [&](auto clear) GDR_INLINE {
        if (role) walk_as(std::integral_constant<int, 1>{}, clear);
        else      walk_as(std::integral_constant<int, 0>{}, clear);
    };
    walk(std::false_type{});
    if (__builtin_expect(__syncthreads_or(R::any_odd(acc)), 0)) walk(std::true_type{});
    if (j >= bl.len) return;
    const size_t to = ((size_t)(bl.row0 + j) * a.Hkv + hk) * D;
    if (role) R::store(static_cast<T *>(a.dk) + to, acc, h, a.scale);
    else      R::store(static_cast<T *>(a.dv) + to, acc, h, 1.f);
}

// Pairs of a workgroup.  Of 128 channels four fill a CU's LDS; of 64, two
// workgroups of two fit, each with barriers of its own (12 sequences of 300 to
// 6,100 tokens, window 512, 16 heads: both kernels 313 us, 351 with four).
template <int D> constexpr int kPairs = D == 128 ? 4 : 2;

// workgroups at a time, by the registers of a wave (queries; keys, of 128 channels
// by the LDS)
template <typename T, int D>
constexpr int kQueries = 256 * (sizeof(T) == 2 ? (D == 128 ? 2 : 3) : (D == 128 ? 1 : 2));
template <typename T, int D> constexpr int kKeys = 256 * (sizeof(T) == 2 && D == 64 ? 2 : 1);

template <typename T, int D>
hipError_t launch(const PromptArgs &a, hipStream_t s) {
    KArgs k{};
    k.a = a;
    k.c = fminf(fmaxf(a.scale * kLog2e, -3.4e38f), 3.4e38f);
    const long long blocks = block_bound<kRows>(a);
    k.lse2 = static_cast<float *>(a.ws);
    k.start = k.lse2 + (size_t)a.Hq * a.T_total;
    hipError_t e;
    if (few_rows<T, D, Pass::kQueries>(a)) {
        e = launch_queries_short(sizeof(T) == 2, D, a, s);
    } else {
        k.mixed = mixed_seqs<T, kRows>(a, a.Hq, kQueries<T, D>);
        query_kernel<T, D><<<(unsigned)(blocks * a.Hq), kThreads, 0, s>>>(k);
        e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
    if (few_rows<T, D, Pass::kKeys>(a)) return launch_keys_short(sizeof(T) == 2, D, a, s);
    if constexpr (sizeof(T) == 2) {
        constexpr int kTokens = 32 * kPairs<D>;
        k.mixed = mixed_seqs<T, kTokens>(a, a.Hkv, kKeys<T, D>);
        key_pairs_kernel<D, kPairs<D>><<<(unsigned)(block_bound<kTokens>(a) * a.Hkv), 4 * kTokens, 0, s>>>(k);
    } else {
        k.mixed = mixed_seqs<T, kRows>(a, a.Hkv, kKeys<T, D>);
        key_kernel<T, D><<<(unsigned)(blocks * a.Hkv), kThreads, 0, s>>>(k);
    }
    return hipGetLastError();
}

}  // namespace

size_t attention_backward_workspace(bool, int, int T_total, int Hq, int, int) {
    return 2 * (size_t)Hq * T_total * sizeof(float);
}

hipError_t launch_attention_backward(bool bf16_io, int D, const PromptArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? launch<bf16, 128>(a, s) : launch<bf16, 64>(a, s);
    return D == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
}

}  // namespace gdr

// prompt.hip -- attention over whole prompts (causal, optionally windowed,
// grouped heads, packed sequences), for gfx950.
//
// Row i of a sequence attends to the tokens j <= i (and j > i - window):
//     s_ij = scale q_i.k_j,   w_ij = e^{s_ij} / sum e^{s_ij},   o_i = sum w_ij v_j.
//
// One pass over K and V with a running maximum m and sum l, in units of
// y = q.k: with c = |scale| log2 e (a negative scale's sign goes into q),
// w = 2^{c y - c m}, l and o multiplied by 2^{c (m - m')} where m grows to m'.
// m is left behind while it is within 2^8 of the maximum, which keeps every
// weight below 2^8 and spares most tiles the multiplication.
//
// A workgroup has 128 rows of a head, 32 a wave, and takes tiles of 64 tokens (32
// in fp32) through LDS, two there, the next on its way straight from memory while
// one is worked on.  S^T = K Q^T gives a lane logits of one row, whose weights are,
// as they lie, the operand of O^T += V^T P^T: only K and V pass through LDS.  Two
// workgroups share a CU, so that one's exponentials run under the other's
// products.
//
// Products bound it.  16 packed prompts of 512 to 8,192 tokens, 32 heads over 8 of
// 128 in bf16: 1,722 to 1,915 us by the card, 0.94 to 1.05 PFLOP/s (a library's product of
// 8192^3: 1.21), the matrix units busy for 55 % of the CUs' cycles at about 1.8
// GHz, no bank conflicts in LDS.  Copies of the kernel without a part of it: without
// barriers 1,755 (of 1,780 to 1,805), without fetches 1,564, without exponentials
// 1,653, with products only 1,320.  8 prompts of 700 to 2,900 tokens in fp32,
// window 1,024, 16 heads of 64: 427 us, the matrix units busy for 76 %.  Measured
// and not kept: 256 rows a workgroup (1,806 us for 1,802), the next tile's logits
// under this one's weights (1,880 for 1,865), a wave's priority raised around its
// products (1,870 for 1,805), products and weights interleaved by force (1,884 for
// 1,867).
#include "prompt_internal.h"

namespace gdr {
namespace {

constexpr int kWaves = 4;                  // waves of a workgroup, 32 rows each
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;

struct KArgs {
    PromptArgs a;
    float c;              // |scale| log2 e, above 0
    float ascale;         // |scale|
    bool negative;        // scale < 0
    int mixed;            // mixed_seqs
};

// waves a SIMD that a wave's registers leave room for
template <typename T, int D>
constexpr int kShare = Rows<T, D>::kRowBytes > 256 ? 1 : Rows<T, D>::kRowBytes > 128 ? 2 : 4;

template <typename T, int D>
__global__ __launch_bounds__(kThreads, (kShare<T, D>)) void prompt_kernel(KArgs k) {
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

    typename R::B q;
    {
        const int row = i < bl.len ? i : bl.len - 1;
        R::load(q, static_cast<const T *>(a.q) + ((size_t)(bl.row0 + row) * a.Hq + head) * D, h);
        if (k.negative) R::negate(q);
    }
    const int last = i0 + kRows < bl.len ? i0 + kRows - 1 : bl.len - 1;
    const int first = a.window > 0 && i0 >= a.window ? i0 - a.window + 1 : 0;
    const int t0 = first / kTok, t1 = last / kTok + 1;

    const unsigned span = a.window > 0 ? a.window : 1u << 31;     // tokens a row attends to
    auto attends = [&](int j) GDR_INLINE { return (unsigned)(i - j) < span; };
    // every row of the wave attends to all of a tile (rows past the sequence's
    // end, which are not stored, among them)
    auto tile_full = [&](int t) GDR_INLINE {
        return t * kTok + kTok - 1 <= iw && (a.window == 0 || t * kTok > iw + 31 - a.window);
    };
    const Fetch<T, D, kWaves> fetch(kpitch, w, lane);
    auto stage = [&](int t) GDR_INLINE {
        const size_t row = (size_t)bl.row0 + t * kTok;
        const int left = bl.len - t * kTok;
        fetch(lds[t & 1][0], kh, row, left, lane);
        fetch(lds[t & 1][1], vh, row, left, lane);
    };
    float m, mc, l;
    unsigned small = 0;                      // rows whose weights are kDown times theirs
    f32x16 acc[kCols];
    // All tiles.  CLEAR: infinities and NaN are taken out of V where some row
    // does not attend to a token, and the weights of `small` rows are made smaller.
    auto walk = [&](auto clear) GDR_INLINE {
        constexpr bool CLEAR = decltype(clear)::value;
        const float down = CLEAR && (small >> r & 1) ? kDown : 1.f;
        m = -INFINITY;
        mc = l = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c][e] = 0.f;
        stage(t0);
        R::settle(q);
        for (int t = t0; t < t1; ++t) {
            tile_landed();
            if (t + 1 < t1) stage(t + 1);
            const int j0 = t * kTok;
            const char *kt = lds[t & 1][0], *vt = lds[t & 1][1];
            // no row of this wave attends to the tile
            if (iw >= bl.len || j0 > iw + 31 || (a.window > 0 && j0 + kTok <= iw - a.window + 1))
                continue;
            f32x16 x[kBlk];
#pragma unroll
            for (int b = 0; b < kBlk; ++b) x[b] = R::rows(kt, b, at, q);
            R::template ahead<kBlk>();
            const bool full = tile_full(t);
            if (!full) {
#pragma unroll
                for (int b = 0; b < kBlk; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[b][e] = attends(j0 + 32 * b + R::key(e, h)) ? x[b][e] : -INFINITY;
            }
            float top = x[0][0];
#pragma unroll
            for (int b = 0; b < kBlk; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, x[b][e]);
            const float mn = fmaxf(m, swap_max32(top));
            const bool grow = (mn - m) * k.c > 8.f;      // (not while both are -inf)
            if (__builtin_amdgcn_ballot_w64(grow)) {
                const float al = grow ? exp2_((m - mn) * k.c) : 1.f;
                l *= al;
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[c] *= al;
                m = grow ? mn : m;
                mc = grow ? mn * k.c : mc;
            }
#pragma unroll
            for (int b = 0; b < kBlk; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[b][e] = exp2_(fmaf(x[b][e], k.c, -mc));
                    if (CLEAR) x[b][e] *= down;
                    l += x[b][e];
                }
#pragma unroll
            for (int b = 0; b < kBlk; ++b)
                R::template cols<CLEAR>(acc, vt, b, at, R::operand(x[b]), full);
        }
    };
    walk(std::false_type{});
    // A weight of zero must not meet an infinity or NaN of V.  Where one has, a
    // result is NaN: then all is done again without such values, and the rows
    // that do attend to them get them after.  Rows whose sums are infinite or NaN
    // even so are summed once more, smaller (the others to the same bits).
    if (__builtin_expect(__syncthreads_or(R::any_odd(acc)), 0)) {
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            walk(std::true_type{});
            if (pass) break;
            small = rows_of(R::any_odd(acc));
            if (!__syncthreads_or(small)) break;
        }
        for (int j = first; j <= last; ++j)
            if (!tile_full(j / kTok) && attends(j))
                R::add_odd(acc, vh + (size_t)(bl.row0 + j) * a.Hkv * D, h);
    }
    if (i >= bl.len) return;
    l = swap_sum32(l);
    const size_t row = (size_t)(bl.row0 + i) * a.Hq + head;
    if (l == 0.f) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c][e] = 0.f;
    }
    R::store(static_cast<T *>(a.o) + row * D, acc, h, l == 0.f ? 0.f : 1.f / l);
    if (a.lse && h == 0)
        a.lse[row] = l == 0.f ? -INFINITY : m * k.ascale + kLn2F * __builtin_amdgcn_logf(small >> r & 1 ? l * kUp : l);
}

// workgroups at a time, by the registers of a wave
template <typename T, int D>
constexpr int kResident = 256 * (sizeof(T) == 2 ? (D == 128 ? 2 : 4) : (D == 128 ? 1 : 3));

template <typename T, int D>
hipError_t launch(const PromptArgs &a, hipStream_t s) {
    KArgs k{};
    k.a = a;
    // (a scale of zero: the smallest number, whose products vanish)
    k.ascale = fabsf(a.scale);
    k.c = fminf(fmaxf(fabsf(a.scale * kLog2e), 1.4e-45f), 3.4e38f);
    k.negative = a.scale < 0.f;
    const long long blocks = block_bound<kRows>(a);
    if (few_rows<T, D, Pass::kForward>(a)) return launch_prompt_short(sizeof(T) == 2, D, a, s);
    k.mixed = mixed_seqs<T, kRows>(a, a.Hq, kResident<T, D>);
    prompt_kernel<T, D><<<(unsigned)(blocks * a.Hq), kThreads, 0, s>>>(k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_prefill(bool bf16_io, int D, const PromptArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? launch<bf16, 128>(a, s) : launch<bf16, 64>(a, s);
    return D == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
}

}  // namespace gdr

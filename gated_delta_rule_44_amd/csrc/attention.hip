// attention.hip -- attention of new tokens over the paged key-value cache,
// for gfx950.
//
// Row (b, t, h) of the queries stands at position p = len_b - n + t and
// attends to the cached tokens j <= p (and j > p - window):
//     s_j = scale q.k_j,   w_j = e^{s_j} / sum e^{s_i},   o = sum w_j v_j.
#include "cache_internal.h"
#include "gdr_internal.h"
#include "device_util.h"

namespace gdr {
namespace {

// First and one past the last token that row t of sequence b attends to
// (empty when lo >= hi).
struct Span { int lo, hi; };
__device__ inline Span row_span(const AttnArgs &a, int len, int t) {
    const int p = len - a.n + t;
    Span s{0, p + 1};
    if (a.window > 0 && p >= a.window) s.lo = p - a.window + 1;
    return s;
}

__device__ inline float wave_sum(float x) {
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

// One workgroup of four waves per query row; a wave takes every fourth token,
// its 64 lanes the D channels, with the running maximum and sum of the
// softmax; the four partial results are joined through LDS.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_row_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const long long row = blockIdx.x;                 // (b, t, hq)
    const int hq = (int)(row % a.Hq);
    const int t = (int)(row / a.Hq % a.n), b = (int)(row / a.Hq / a.n);
    const int h = hq / a.G;
    const T *q = static_cast<const T *>(a.q) + row * D;
    const T *kc = static_cast<const T *>(a.k_cache), *vc = static_cast<const T *>(a.v_cache);
    const int len = cached_len(a.seq_lens, b, a.map);
    const Span sp = row_span(a, len, t);
    float qv[E], acc[E] = {};
    for (int e = 0; e < E; ++e) qv[e] = Elem<T>::load(q + lane * E + e) * a.scale;
    float m = -INFINITY, z = 0.f;
    for (int j = sp.lo + w; j < sp.hi; j += 4) {
        const int page = page_of(a.map, b, j);
        if (page < 0) continue;
        const size_t at = cache_row(a.map, a.Hkv, page, h, slot_of(a.map, j)) * D + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += qv[e] * Elem<T>::load(kc + at + e);
        s = wave_sum(s);
        const float mn = fmaxf(m, s), mm = mn == -INFINITY ? 0.f : mn;
        const float c = expf(m - mm), p = expf(s - mm);
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + p * Elem<T>::load(vc + at + e);
        z = z * c + p;
        m = mn;
    }
    __shared__ float sm[4], sz[4], sacc[4][D];
    sm[w] = m; sz[w] = z;
    for (int e = 0; e < E; ++e) sacc[w][lane * E + e] = acc[e];
    __syncthreads();
    if (w > 0) return;
    float mt = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float mm = mt == -INFINITY ? 0.f : mt;
    float zt = 0.f, at[E] = {};
    for (int i = 0; i < 4; ++i) {
        const float c = expf(sm[i] - mm);
        zt += sz[i] * c;
        for (int e = 0; e < E; ++e) at[e] += sacc[i][lane * E + e] * c;
    }
    T *o = static_cast<T *>(a.o) + row * D;
    for (int e = 0; e < E; ++e) Elem<T>::store(o + lane * E + e, zt == 0.f ? 0.f : at[e] / zt);
    if (a.scores && lane == 0) {
        static_cast<float *>(a.ws)[2 * row] = mm;
        static_cast<float *>(a.ws)[2 * row + 1] = zt;
    }
}

// The weights of every row that reads a token, summed in the rows' order:
// one wave per (sequence, head, token).
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_score_kernel(AttnArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int bh = blockIdx.y, b = bh / a.Hkv, h = bh % a.Hkv;
    const int j = blockIdx.x * 4 + w;
    const int len = cached_len(a.seq_lens, b, a.map);
    if (j >= len) return;
    const int page = page_of(a.map, b, j);
    if (page < 0) return;
    const size_t cr = cache_row(a.map, a.Hkv, page, h, slot_of(a.map, j));
    const T *kc = static_cast<const T *>(a.k_cache) + cr * D + lane * E;
    float sum = 0.f;
    for (int t = 0; t < a.n; ++t) {
        const Span sp = row_span(a, len, t);
        if (j < sp.lo || j >= sp.hi) continue;
        for (int g = 0; g < a.G; ++g) {
            const long long row = ((long long)b * a.n + t) * a.Hq + h * a.G + g;
            const T *q = static_cast<const T *>(a.q) + row * D + lane * E;
            float s = 0.f;
            for (int e = 0; e < E; ++e) s += Elem<T>::load(q + e) * a.scale * Elem<T>::load(kc + e);
            s = wave_sum(s);
            const float *st = static_cast<const float *>(a.ws) + 2 * row;
            if (st[1] != 0.f) sum += expf(s - st[0]) / st[1];
        }
    }
    if (lane == 0) a.scores[cr] += sum;
}

template <typename T, int D>
hipError_t launch(const AttnArgs &a, hipStream_t s) {
    attn_row_kernel<T, D><<<(unsigned)((long long)a.B * a.n * a.Hq), 256, 0, s>>>(a);
    const int cap = a.map.max_pages << a.map.page_shift;
    if (a.scores && cap > 0)
        attn_score_kernel<T, D><<<dim3((cap + 3) / 4, a.B * a.Hkv), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int B, int n, int Hq, int Hkv, int D, long long capacity,
                           bool with_scores) {
    (void)Hkv; (void)D; (void)capacity;
    return with_scores ? (size_t)B * n * Hq * 2 * sizeof(float) : 0;
}

hipError_t launch_attention_decode(bool bf16_io, int D, const AttnArgs &a, hipStream_t s) {
    if (bf16_io) return D == 128 ? launch<bf16, 128>(a, s) : launch<bf16, 64>(a, s);
    return D == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
}

}  // namespace gdr
